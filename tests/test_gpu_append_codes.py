"""The codes of an 8-bit cache, each of them: E4M3 of the exact quotient value /
scale, nearest, ties to the even code, saturated at 448 (GB300 only).

The quotient of an fp32 value and an fp32 scale that is not itself halfway
between two codes is at least 2^-29 of its size away from there (the numerator
minus the 5-bit halfway point times the 24-bit scale is a whole number of units
of 2^-29 of it), so the quotient in 64 bits, off by 2^-53, tells the side."""
import numpy as np
import pytest
import torch

from test_gpu_rope import DEV, T, gen

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import row_reduction_norm_gb300 as R

CODES = np.arange(127)                                    # of values >= 0
EXP, MAN = CODES >> 3, CODES & 7
VALUES = np.where(EXP > 0, (8 + MAN) * 2.0 ** (EXP - 10.0), MAN * 2.0 ** -9)
HALFWAY = (VALUES[1:] + VALUES[:-1]) / 2


def codes_of(v, scale):
    """The codes of an fp32 tensor's values, a numpy array of bytes."""
    x = v.float().cpu().numpy()
    with np.errstate(all="ignore"):
        q = np.abs(x.astype(np.float64) / float(np.float32(scale)))
    low = np.searchsorted(HALFWAY, q, side="left")        # halfway points below q
    tie = (low < 126) & (q == HALFWAY[np.minimum(low, 125)])
    code = np.where(tie & (low % 2 == 1), low + 1, low)
    code = np.where(np.isnan(x), 127, code)
    return (code + 128 * np.signbit(x)).astype(np.uint8)


def append(x, d, rot, scale, k_heads):
    """Rows of [keys | values], stored as they are (no norm, position 0): the
    keys' and the values' codes."""
    rows = x.shape[0]
    dev = x.device
    kc, vc = (torch.zeros(rows, 1, k_heads, d, device=dev).to(torch.float8_e4m3fn) for _ in range(2))
    table = torch.arange(rows, device=dev, dtype=torch.int32)[None].contiguous()
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
    f = torch.ones(rot // 2, device=dev)
    R.qkv_append(x, kc, vc, table, ints(0, rows), ints(0), 0, k_heads, d, f, norm=False, k_scale=scale, v_scale=scale,
                 positions=torch.zeros(rows, dtype=torch.int64, device=dev))
    return (c.view(torch.uint8).reshape(rows, -1).cpu().numpy() for c in (kc, vc))


SCALES = [0.05, 0.03, 1 / 3, 0.0123456, 1.7, 113.0, 1.0, 0.0625, 2.0 ** -100, 2.0 ** 100, 1.3e-30, 7e29,
          float(np.float32(448.0) / np.float32(57344.0)), 0.9999999]


# heads in whole pieces, through shared memory, in single elements
@pytest.mark.parametrize("d,rot", [(128, 128), (80, 20), (34, 34), (64, 48)])
@pytest.mark.parametrize("scale", SCALES)
def test_codes_of_every_bf16_value(d, rot, scale):
    """Every bf16 number; NaN codes are compared as NaN."""
    k = 2
    row = 2 * k * d
    n = -(-65536 // (k * d))
    half = torch.arange(n * k * d, device=DEV).remainder(65536).to(torch.int32)
    half = half.to(torch.int16).view(torch.bfloat16).view(n, k * d)
    # a rotation by 0 of a pair with an infinity or NaN in it is not the identity
    keys = torch.where(half.isfinite(), half, torch.zeros_like(half))
    x = torch.cat((keys, half), 1)
    assert x.shape[1] == row
    for got, v, what in zip(append(x, d, rot, scale, k), (keys, half), ("keys", "values")):
        want = codes_of(v, scale)
        if what == "keys":      # 0 - 0 turns -0 into 0
            got, want = np.where(got == 128, 0, got), np.where(want == 128, 0, want)
        both = ((got & 127) == 127) & ((want & 127) == 127)
        bad = (got != want) & ~both
        assert not bad.any(), (what, int(bad.sum()), float(v.cpu()[tuple(np.argwhere(bad)[0])]), int(got[bad][0]),
                               int(want[bad][0]))


@pytest.mark.parametrize("d,rot", [(128, 128), (80, 20), (34, 34)])
def test_codes_next_to_the_halfway_points(d, rot):
    """fp32 values whose quotient lies at a halfway point or within three steps of one."""
    k, g = 1, gen(d)
    for scale in SCALES:
        s = np.float32(scale)
        at = (HALFWAY * float(s)).astype(np.float32)
        at = np.concatenate([at, VALUES.astype(np.float32) * s])
        near = np.concatenate([(at.view(np.int32) + i).view(np.float32) for i in range(-3, 4)])
        near = np.concatenate([near, -near])
        near = near[np.isfinite(near)]
        pad = -len(near) % (k * d)
        v = torch.from_numpy(np.concatenate([near, np.zeros(pad, np.float32)])).to(DEV).view(-1, k * d)
        x = torch.cat((v, v), 1)
        for got, what in zip(append(x, d, rot, scale, k), ("keys", "values")):
            want = codes_of(v, scale)
            got, want = np.where(got == 128, 0, got), np.where(want == 128, 0, want)
            bad = got != want
            assert not bad.any(), (what, scale, int(bad.sum()), float(v.cpu()[tuple(np.argwhere(bad)[0])]),
                                   int(got[bad][0]), int(want[bad][0]))
