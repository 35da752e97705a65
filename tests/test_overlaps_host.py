"""Calls whose outputs share memory with what they read or write elsewhere are refused on the host (no GPU, no kernel launched:
every call below is refused).  Rows are laid out by brute force, cell by cell, beside the library's arithmetic."""
import random

from test_block_ops_host import A, ARG, BF16, FP32, GRAD, RES, back, dual, quant, residual, rotary

ES = {BF16: 2, FP32: 4}


def rows_of(p, n, ld, columns, es):
    return {(p // es + i * ld) * es + b for i in range(n) for c in range(columns) for b in range(c * es, c * es + es)}


# bytes of each operand of a call on RES / GRAD's shapes
def sizes(base, **more):
    T, C = base["T"], base["C"]
    matrix, vector, stat = 2 * T * C, 2 * C, 4 * T
    return {**{k: matrix for k in ("h", "x", "h_out", "y", "dy", "dh_out", "dh", "dx")}, **{k: vector for k in ("weight", "bias", "gate", "post_weight")},
            **{k: stat for k in ("mean", "rstd", "post_mean", "post_rstd")}, **{k: 4 * C for k in ("dweight", "dbias", "dgate", "dpost_weight")}, **more}


def ends(base, size, align):
    """Places at which `size` bytes overlap those of `base` = (address, bytes): their ends by one unit, and the middle."""
    at, n = base
    up = lambda v: -(-v // align) * align
    return {up(at - size + align) if size > align else at, at, at + up(n) - align if up(n) > align else at}


def clashes(call, place, size, read, written, align, free):
    """Every written operand over every other one (free: pairs that may be the same tensor, at the same place)."""
    for out in written:
        for other in (*read, *written):
            if other == out:
                continue
            for at in ends((place[other], size[other]), size[out], align):
                if at == place[other] and (out, other) in free:
                    continue
                assert call(**{out: at}) == ARG, (out, other, at - place[other])


IN, STATS = ("h", "x", "weight", "bias", "gate", "post_weight"), ("mean", "rstd", "post_mean", "post_rstd")
REPLACED = {(o, i) for o in ("h_out", "y") for i in ("h", "x")}


def test_residual():
    clashes(residual, {**RES, "y": A[11]}, sizes(RES), IN, ("h_out", "y", *STATS), 4, REPLACED)
    for T in (2, 4):                                                 # in place, but with another stride
        for out, given in REPLACED:
            ld = {"y": "ldy", "h_out": "ldh_out"}[out]
            assert residual(**{"T": T, out: RES[given], ld: 264}) == ARG
    assert residual(h_out=RES["h"], y=RES["h"]) == ARG and residual(h_out=RES["x"], y=RES["x"]) == ARG


def test_residual_codes():
    size = sizes(RES, q=4 * 256, s=4 * 2 * 4)
    clashes(quant, {**RES, "q": A[11], "s": A[12]}, size, IN, ("h_out", "q", "s"), 16, REPLACED)
    size = sizes({**RES, "T": 256}, q=256 * 256, s=4 * 2 * 256, qT=256 * 256, sT=4 * 2 * 256)
    clashes(dual, {**RES, "q": A[11], "s": A[12], "qT": A[13], "sT": A[14]}, size, IN,
            ("h_out", "q", "s", "qT", "sT", "mean", "rstd"), 16, REPLACED)


def test_residual_backward():
    place = {**GRAD, "dbias": A[13] + 8192, "ws": 1 << 36}
    read = ("dy", "h_out", "dh_out", "x", "weight", "gate", "post_weight", *STATS)
    written = ("dh", "dx", "dweight", "dbias", "dgate", "dpost_weight")
    free = {(o, i) for o in ("dh", "dx") for i in ("dy", "h_out", "dh_out", "x")}
    call = lambda **k: back(**{"dbias": place["dbias"], "ws": place["ws"], **k})
    clashes(call, place, sizes(GRAD), read, written, 4, free)
    from blockwise_scaled_fp8_quant_amd import puro_residual_norm_backward_workspace_size as need
    assert need(64, 256, True) > 0
    for other in (*read, *written):                                  # the workspace over anything
        assert call(ws=place[other] // 16 * 16) == ARG and call(ws=place[other] - need(64, 256, True) + 16) == ARG, other
    for out, ld in (("dh", "lddh"), ("dx", "lddx")):
        for given in ("dy", "h_out", "dh_out", "x"):
            assert call(**{out: place[given], ld: 264}) == ARG, (out, given)
    assert call(dh=place["dy"], dx=place["dy"]) == ARG


def test_rows_that_interleave():
    """h_out laid over h in one buffer with strides of its own: refused where a cell is in both."""
    rng = random.Random(3)
    base, seen = 1 << 33, 0
    for _ in range(4000):
        T, C = rng.randint(1, 6), rng.randint(1, 8)
        ld = C + rng.randint(0, 12)
        other = ld if rng.random() < 0.5 else C + rng.randint(0, 20)
        at = base + 4 * rng.randint(0, 80)
        if at == base and (T == 1 or ld == other):
            continue
        if rows_of(at, T, other, C, 4) & rows_of(base, T, ld, C, 4):
            seen += 1
            assert residual(x_dtype=FP32, T=T, C=C, h=base, ldh=ld, ldx=C, h_out=at, ldh_out=other, ldy=C) == ARG, (T, C, ld, other, at - base)
    assert seen > 1000


def heads_of(p, T, H, D, ld_t, ld_h):
    return {p + i * ld_t + k * ld_h + d for i in range(T) for k in range(H) for d in range(D)}


def apart(T, H, D, ld_t, ld_h):
    return len(heads_of(0, T, H, D, ld_t, ld_h)) == T * H * D and (T == 1 or ld_t >= D) and (H == 1 or ld_h >= D)


def test_rotary_heads_that_interleave():
    """x and y in one buffer, tokens or heads outermost, strides alike or their own, x's heads over each other too."""
    rng = random.Random(4)
    base, seen, alike = 1 << 33, 0, 0
    while seen < 3000:
        T, H, D = rng.randint(1, 4), rng.randint(1, 4), rng.randint(1, 6)
        inner = D + rng.randint(0, 8)
        outer = (max(T, H) - 1) * inner + D + rng.randint(0, 20)
        ldy = (outer, inner) if rng.random() < 0.5 else (inner, outer)
        if not apart(T, H, D, *ldy):
            continue
        ldx = ldy if rng.random() < 0.5 else (rng.randint(0, 30), rng.randint(0, 30))
        at = rng.randint(0, 100) if rng.random() < 0.9 else 0
        same = (T == 1 or ldx[0] == ldy[0]) and (H == 1 or ldx[1] == ldy[1])
        if (at == 0 and same) or not heads_of(at, T, H, D, *ldx) & heads_of(0, T, H, D, *ldy):
            continue
        seen += 1
        alike += ldx == ldy
        assert rotary(xd=FP32, x=base + 4 * at, ld_t=ldx[0], ld_h=ldx[1], T=T, H=H, D=D, pairs=0, y=base, ldy_t=ldy[0], ldy_h=ldy[1]) == ARG, \
            (T, H, D, ldx, ldy, at)
    assert 500 < alike < 2500


def test_rotary_positions_and_frequencies():
    """4 tokens of 4 heads of 128 in bf16: 4096 bytes at A[3]; 32 of positions, 512 of frequencies."""
    for at in (A[3] - 24, A[3], A[3] + 2048, A[3] + 4088):
        assert rotary(pos=at) == ARG
    for at in (A[3] - 504, A[3], A[3] + 4088):
        assert rotary(freqs=at) == ARG
    assert rotary(x=A[3] + 2) == ARG and rotary(x=A[3] + 4094) == ARG and rotary(x=A[3] - 4094) == ARG
    # between y's heads there is room for a head, not for one and a value
    assert rotary(x=A[3] + 2 * 126, ld_t=1024, ld_h=256, ldy_t=1024, ldy_h=256) == ARG
    assert rotary(x=A[3] + 2 * 130, ld_t=1024, ld_h=256, ldy_t=1024, ldy_h=256) == ARG
