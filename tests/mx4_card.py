"""What tests of the MXFP4 operators on the card share: random matrices with their values
in 64 bits, rows, and the comparison by the tolerances of test_gpu_mx4.py."""
import torch

ROUND = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}
DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def matrix(qp, g, *shape, scales=(118, 130)):
    """A random MX4 with scales of a range, and its values in f64 on the card."""
    *lead, K = shape
    G = -(-K // 32)
    codes = torch.randint(0, 256, (*lead, 16 * G), generator=g, dtype=torch.uint8)
    if K % 32:  # the values past K are zeros
        both = torch.stack((codes & 15, codes >> 4), -1).reshape(*lead, 32 * G)
        both[..., K:] = 0
        codes = both[..., 0::2] | (both[..., 1::2] << 4)
    s = torch.randint(*scales, (*lead, G), generator=g, dtype=torch.uint8)
    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)
    grid = torch.cat((grid, -grid))
    v = grid[torch.stack((codes & 15, codes >> 4), -1).long()].reshape(*lead, 32 * G)
    v = v * torch.pow(2.0, s.double() - 127).repeat_interleave(32, -1)
    return qp.mx4_tensor(codes.cuda(), s.cuda(), K), v[..., :K].cuda()


def rows(x, dtype, odd):
    """Rows x of K + 3 columns as K of the type, at an odd address or not; and in f64."""
    x, K = x.to(DTYPE[dtype]).cuda(), x.shape[1] - 3
    x = x[:, 1:1 + K] if odd else x[:, :K].contiguous()
    return x, x.double()


def close(got, want, A, terms, dtype, what):
    """A: the sums of the terms' magnitudes."""
    got = got.double()
    assert torch.isfinite(got).all(), what
    tol = (3 * terms / 32 + 64) * 2.0 ** -23 * A + ROUND[dtype] * want.abs() * 1.01 \
        + (2.0 ** -25 if dtype == "f16" else 0.0)
    off = (got - want).abs()
    assert (off <= tol).all(), "%s: %d outputs off, worst by %.3g of its tolerance" % (
        what, int((off > tol).sum()), float((off / tol.clamp_min(1e-300)).max()))


def t(w):
    """The transpose, laid out anew (for batched products of torch)."""
    return w.transpose(-1, -2).contiguous()
