"""Runs the 8-bit products' kernels under the checked build (started by
test_gpu_checked_fp8.py with TMAGEMM_CHECKED=1): after each call no self-check
may have fired, every work unit must have completed exactly once, and the
integer-valued result must be exact.  Exits non-zero on the first failure."""
import json
import os

import torch

assert os.environ.get("TMAGEMM_CHECKED") == "1"
import tma_pipelined_tensor_tn_gb300 as tg  # noqa: E402

tg.build()
assert tg.CHECKED
gen = torch.Generator(device="cuda").manual_seed(0)


def ints(*shape):
    v = torch.randint(-4, 5, shape, device="cuda", generator=gen)
    return v.float(), v.float().to(torch.float8_e4m3fn)


def verify(name, got, want, units=None):
    st = tg.lib().tmagemm_check(None)
    assert st == tg.TMAGEMM_OK, (name, tg.strerror(st), tg.tmagemm_last_error_detail())
    counts = tg.checked_unit_counts(8192)
    done = sum(counts)
    assert done > 0 and all(c == 1 for c in counts[:done]), (name, done, max(counts))
    assert units is None or done in units, (name, done, units)
    assert torch.equal(got.float(), want.to(got.dtype).float()), name
    print(json.dumps({"case": name, "units": done}), flush=True)


def div(a, b):
    return -(-a // b)


for M, N, K in ((1, 4096, 4112), (16, 136, 144), (40, 14336, 400), (100, 1000, 528),
                (256, 512, 4096), (777, 2056, 528), (1237, 5000, 272), (2048, 4096, 272),
                (4096, 4096, 400)):
    a, qa = ints(M, K)
    b, qb = ints(N, K)
    d = tg.gemm_fp8(qa, torch.ones((M, div(K, 128)), device="cuda"), qb,
                    torch.ones((div(N, 128), div(K, 128)), device="cuda"))
    units = None
    if M > 256:
        units = [div(M, 256) * div(N, n) for n in (192, 256)] + [div(M, 128) * div(N, 128)]
    verify(f"dense_{M}x{N}x{K}", d, a @ b.t(), units)

for counts in ([0, 1, 129, 0, 16, 17, 300], [700, 513, 0, 1, 256], [2] * 64):
    N, K, G, M = 1000, 272, len(counts), sum(counts)
    off = [0]
    for c in counts:
        off.append(off[-1] + c)
    a, qa = ints(M, K)
    b, qb = ints(G, N, K)
    d = tg.gemm_fp8_grouped(qa, torch.ones((M, 3), device="cuda"), qb,
                            torch.ones((G, 8, 3), device="cuda"),
                            torch.tensor(off, dtype=torch.int32, device="cuda"))
    want = torch.cat([a[off[g]:off[g + 1]] @ b[g].t() for g in range(G)])
    units = [sum(div(c, tm) for c in counts) * div(N, tn)
             for tm, tn in ((128, 128), (256, 192), (256, 256))]
    verify(f"grouped_{G}_{M}", d, want, units)
print("CHECKED OK", flush=True)
