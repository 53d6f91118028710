"""Shapes that reach every form of the adapters' kernels, and their reference on
the GPU in 64 bits."""
import torch

# (T, n, r, K, N)
FORMS = [
    # up to 64 rows: decode batches of many adapters and of few, wide outputs
    (17, 1, 8, 72, 30), (17, 1, 40, 72, 30), (64, 64, 64, 512, 300), (64, 64, 24, 136, 30), (64, 1, 168, 264, 30),
    (63, 12, 72, 72, 30), (33, 2, 8, 72, 66000), (64, 1, 40, 72, 66000), (64, 1, 72, 72, 33000), (64, 1, 248, 72, 33000),
    (64, 1, 72, 72, 44000), (64, 1, 136, 72, 44000), (64, 1, 8, 72, 131072), (64, 1, 64, 72, 131080),
    # more rows
    (65, 1, 8, 72, 30), (65, 1, 40, 72, 30), (96, 1, 104, 264, 30), (96, 1, 200, 72, 30), (512, 32, 64, 512, 700),
    (130, 8, 8, 72, 20000), (65, 1, 40, 72, 66000), (320, 1, 72, 72, 11000), (320, 1, 136, 72, 11000),
    (65, 2, 8, 72, 66000), (65, 2, 40, 72, 66000), (512, 3, 72, 264, 11000), (384, 1, 200, 72, 17000),
    (512, 8, 128, 512, 8192), (200, 4, 256, 264, 17408), (512, 8, 64, 72, 17408),
]


def adapters(T, n, r, K, N, dtype, seed):
    """y, x, a, b, adapter, scales on the GPU; some rows without an adapter."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    y, x = torch.randn((T, N), generator=g, device="cuda"), torch.randn((T, K), generator=g, device="cuda").to(dtype)
    a = (torch.randn((n, r, K), generator=g, device="cuda") * K ** -0.5).to(dtype)
    b = (torch.randn((n, N, r), generator=g, device="cuda") * r ** -0.5).to(dtype)
    adapter = torch.randint(-1, n, (T,), generator=g, device="cuda", dtype=torch.int32)
    return y, x, a, b, adapter, 0.5 + torch.rand(n, generator=g, device="cuda")


def reference(y, x, a, b, adapter, scales=None):
    """(out, tolerance) in fp64.  The bound counts:
    * K products of 16-bit values (exact) summed in fp32 in any order, K + 8
      roundings of the sum of their sizes;
    * the rank's sums in 16-bit parts: bf16 three, which have all their 24 bits;
      fp16 two, within 2^-23 of the row's largest;
    * r times as many products summed in fp32, 3 r + 8 roundings of the sum of
      their sizes (which the parts make up to 2^-8 larger);
    * the scale and the sum with y, 3 roundings."""
    out = y.double()
    tol = torch.zeros_like(out)
    K, r = x.shape[1], a.shape[1]
    for i in range(a.shape[0]):
        rows = (adapter == i).nonzero()[:, 0]
        if not rows.numel():
            continue
        s = 1.0 if scales is None else float(scales[i])
        xi, ai, bi = x[rows].double(), a[i].double().T.contiguous(), b[i].double().T.contiguous()
        v = xi @ ai
        out[rows] += s * (v @ bi)
        down, up = (xi.abs() @ ai.abs()) @ bi.abs(), 1.01 * (v.abs() @ bi.abs())
        tol[rows] += abs(s) * ((K + 8) * 2.0 ** -24 * down + (3 * r + 8) * 2.0 ** -24 * up)
        if x.dtype == torch.float16:
            tol[rows] += abs(s) * 2.0 ** -23 * v.abs().amax(1, keepdim=True) * bi.abs().sum(0)
    return out, tol + 3 * 2.0 ** -24 * (y.double().abs() + out.abs())


def whole_numbers(T, n, r, K, dtype, seed):
    """y = 0, x, a, b, adapter and the rank's sums v [T, r], on the CPU: sums of
    24 bits, whole numbers that fp32 adds up exactly in any order, of which b
    takes one to each column."""
    g = torch.Generator().manual_seed(seed)
    lo = int((2 ** 23 / K) ** 0.5) + 1  # sums from 2^23 on ..
    hi = int(((2 ** 24 - 1) / K) ** 0.5)  # .. to below 2^24
    assert lo < hi <= 256  # which bf16 has all
    x = torch.randint(lo, hi + 1, (T, K), generator=g)
    a = torch.randint(lo, hi + 1, (n, r, K), generator=g)
    adapter = torch.randint(0, n, (T,), generator=g, dtype=torch.int32)
    v = torch.stack([a[int(i)] @ row for i, row in zip(adapter, x)])
    assert int(v.min()) >= 2 ** 23 and int(v.max()) < 2 ** 24
    b = torch.eye(r).expand(n, r, r).contiguous()
    return torch.zeros(T, r), x.to(dtype), a.to(dtype), b.to(dtype), adapter, v
