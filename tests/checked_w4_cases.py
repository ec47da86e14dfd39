"""Runs the products with 4-bit weights under the checked build (started by
test_gpu_checked_w4.py with TMAGEMM_CHECKED=1): after each call no self-check may have fired,
every work unit must have completed exactly once, and the whole-valued result must be exact.
Exits non-zero on the first failure."""
import json
import os

import torch

assert os.environ.get("TMAGEMM_CHECKED") == "1"
import tma_pipelined_tensor_tn_gb300 as tg  # noqa: E402

tg.build()
assert tg.CHECKED
gen = torch.Generator(device="cuda").manual_seed(0)


def weights(*shape):
    b = torch.randint(0, 256, (*shape[:-1], shape[-1] // 2), device="cuda", generator=gen)
    q = torch.stack((b & 15, b >> 4), dim=-1).flatten(-2) - 8
    return b.to(torch.uint8), q.double()


def verify(name, got, want):
    st = tg.lib().tmagemm_check(None)
    assert st == tg.TMAGEMM_OK, (name, tg.strerror(st), tg.tmagemm_last_error_detail())
    counts = tg.checked_unit_counts(8192)
    done = sum(counts)
    assert done > 0 and all(c == 1 for c in counts[:done]), (name, done, max(counts))
    assert torch.equal(got, want.to(got.dtype)), name
    print(json.dumps({"case": name, "units": done}), flush=True)


# Tokens of 0 and powers of two, few enough that no sum passes 2^8 of the least.
def tokens(M, K):
    a = torch.zeros((M, K), device="cuda")
    at = torch.randint(0, K, (M, 8), device="cuda", generator=gen)
    return a.scatter_(1, at, 1.0)


for dtype in (torch.float16, torch.bfloat16):
    for M, N, K, group in ((1, 4096, 2048, 128), (5, 333, 544, 32), (8, 20000, 256, 64),
                           (9, 128, 32, 32), (16, 4096, 4096, 128), (27, 5003, 2080, 32),
                           (32, 300, 8224, 64), (100, 1000, 1056, 128)):
        a, (b, q) = tokens(M, K), weights(N, K)
        s = torch.ones((N, -(-K // group)), device="cuda", dtype=dtype)
        verify(f"dense_{M}x{N}x{K}", tg.gemm_w4(a.to(dtype), b, s, group=group),
               a.double() @ q.t())
    for counts in ([0, 1, 12, 0, 3], [2] * 64, [40, 0, 9, 70], [8, 100]):
        N, K, G, M = 520, 1312, len(counts), sum(counts)
        off = [0]
        for c in counts:
            off.append(off[-1] + c)
        a, (b, q) = tokens(M, K), weights(G, N, K)
        s = torch.ones((G, N, K // 32), device="cuda", dtype=dtype)
        d = tg.gemm_w4_grouped(a.to(dtype), b, s,
                               torch.tensor(off, dtype=torch.int32, device="cuda"), group=32)
        verify(f"grouped_{G}_{M}", d,
               torch.cat([a[off[g]:off[g + 1]].double() @ q[g].t() for g in range(G)]))
print("CHECKED OK", flush=True)
