"""The bounds of tests/decode_reference.py for weights held in parts can tell them from weights that lost a part: the same
attention in 64 bits with its weights rounded as one or several 16- or 8-bit values, on the inputs that the GPU tests use."""
import numpy as np
import pytest

import decode_reference as ref

torch = pytest.importorskip("torch")

TYPE = {"bf16": torch.bfloat16, "f16": torch.float16}


def rounded(x, dtype):
    return torch.from_numpy(x).float().to(dtype).double().numpy()


def in_parts(p, kind, parts=2):
    up = {"bf16": 1.0, "bf16 planes": 1.0, "f16": 2.0 ** 15, "f16 tensor": 2.0 ** 12}[kind]
    t = TYPE[kind.split()[0]]
    total, left = 0.0, p * up
    for _ in range(parts + (kind == "bf16 planes")):
        x = rounded(left, t)
        total, left = total + x, left - x
    return total / up


def codes(p, n):
    total, left, at = 0.0, p * 32, 32.0
    for k in range(n):
        if k == 2 and n == 4:
            left = rounded(left, torch.float16)
        c = rounded(left, torch.float8_e4m3fn)
        total, left, at = total + c / at, (left - c) * 32, at * 32
    return total


def codes_wide(p):
    """Four codes, the second in the first one's scale."""
    total, left, at = 0.0, p * 32, 32.0
    for k, spacing in enumerate((1, 1024, 32, 1)):
        if k == 2:
            left = rounded(left, torch.float16)
        c = rounded(left, torch.float8_e4m3fn)
        total, left, at = total + c / at, (left - c) * spacing, at * spacing
    return total


@pytest.mark.parametrize("parts", sorted(ref.PARTS))
def test_what_the_parts_leave(parts):
    """Weights of all sizes, up to the 2^3 that the maximum may lag behind."""
    rng = np.random.default_rng(0)
    p = np.concatenate([2.0 ** rng.uniform(-36, 0, 200000), np.float32(2.0) ** -np.arange(36), 1 - 2.0 ** -np.arange(1, 24)])
    p = p.astype(np.float32).astype(np.float64)
    hold = codes_wide if "wide" in parts else (lambda x: codes(x, int(parts[0]))) if "codes" in parts else lambda x: in_parts(x, parts)
    for lag in (1.0, 8.0) if "codes" in parts else (1.0,):
        unit, step, low_unit, low_step = (*ref.PARTS[parts], 0.0, 0.0)[:4]
        off = np.abs(hold(p * lag) / lag - p)
        assert (off <= unit * p + step / lag + np.minimum(low_unit * p, low_step / lag)).all()


def worst(q, k, v, scale, io, parts, hold):
    """Largest |error| / bound of the attention with weights as `hold` makes them."""
    o, l, weight, spread, floor = ref.attend(q, k, v, scale)
    b, _ = ref.parts_bounds(o, l, weight, spread, floor, q.shape[1], len(k), io, parts)
    s = q @ k.T * scale
    p = np.exp(s - s.max(1, keepdims=True))
    got = rounded(hold(p) @ v / p.sum(1, keepdims=True), TYPE[io])
    return (np.abs(got - o) / b).max()


def paired(spread, n=6):
    rng = np.random.default_rng(3)
    k, v = ref.paired_values(rng, n, 1, 64, spread)
    return rng.standard_normal((16, 64)), k[:, 0], v[:, 0]


@pytest.mark.parametrize("spread", [0.3, 0.02, 0.002])
@pytest.mark.parametrize("io,kind", [("bf16", "bf16"), ("f16", "f16"), ("bf16", "f16"), ("f16", "f16 tensor"), ("bf16", "bf16 planes")])
def test_a_lost_second_part_shows(io, kind, spread):
    q, k, v = paired(spread)
    assert worst(q, k, v, 0.125, io, kind, lambda p: in_parts(p, kind)) <= 1
    if kind == "bf16 planes":                                              # of three values: the last one's loss is beside the output's rounding
        assert worst(q, k, v, 0.125, io, kind, lambda p: in_parts(p, kind, 0)) > 1
    elif spread < 0.1 or kind == io:
        assert worst(q, k, v, 0.125, io, kind, lambda p: in_parts(p, kind, 1)) > 1


@pytest.mark.parametrize("n,io", [(3, "bf16"), (3, "f16")])
def test_a_lost_code_shows(n, io):
    """A fourth one of nearly equal weights would not: 2^-14 is beside the output's own rounding."""
    q, k, v = paired(0.002)
    assert worst(q, k, v, 0.125, io, f"{n} codes", lambda p: codes(p, n)) <= 1
    assert worst(q, k, v, 0.125, io, f"{n} codes", lambda p: codes(p, n - 1)) > 1


@pytest.mark.parametrize("gap", [16, 18, 24])
@pytest.mark.parametrize("io,kind", [("f16", "f16"), ("bf16", "f16"), ("f16", "f16 tensor"), ("bf16", "bf16")])
def test_lost_small_weights_show(io, kind, gap):
    """Weights far below the largest one: as f16 values that are not brought up first, they are lost."""
    rng = np.random.default_rng(4)
    k, v = ref.one_large_score(rng, 8193, 1, 64, gap, 0.125, 8.0, 1000.0)
    q = rng.standard_normal((4, 64))
    q[:, 0] = 8.0
    args = q, k[:, 0], v[:, 0], 0.125, io, kind
    assert worst(*args, lambda p: in_parts(p, kind)) <= 1
    if kind != "bf16" and gap > 16:
        assert worst(*args, lambda p: rounded(p, torch.float16)) > 1


@pytest.mark.parametrize("n", [3, 4, "wide"])
def test_lost_small_weights_of_codes_show(n):
    """Four codes hold weights of 2^-26, three are at their end there, as the bound says."""
    rng = np.random.default_rng(4)
    k, v = ref.one_large_score(rng, 8193, 1, 64, 18, 0.125, 8.0, 1.0)
    q = rng.standard_normal((4, 64))
    q[:, 0] = 8.0
    args = q, k[:, 0], v[:, 0], 0.125, "bf16"
    if n == "wide":
        assert worst(*args, "4 codes, wide", codes_wide) <= 1
        assert worst(*args, "4 codes, wide", lambda p: codes(p, 3)) > 1
        return
    assert worst(*args, f"{n} codes", lambda p: codes(p, n)) <= 1
    if n == 4:
        assert worst(*args, f"{n} codes", lambda p: codes(p, n - 1)) > 1


@pytest.mark.parametrize("n,left", [(2, -22), (3, -27)])
def test_what_a_querys_codes_leave(n, left):
    """bf16 elements of a row whose largest is brought into [2^7, 2^8): what n codes leave of them, in units of the largest."""
    x = torch.arange(1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    x = x[torch.isfinite(x) & (x < 256)].double().numpy()
    rest, at, got = x, 1.0, 0.0
    for _ in range(n):
        c = rounded(rest, torch.float8_e4m3fn)
        got, rest, at = got + c / at, (rest - c) * 32, at * 32
    assert np.abs(got - x).max() <= 2.0 ** (7 + left)
    assert (got == x)[x >= 2.0 ** (8 - (14 if n == 2 else 18))].all()
