"""The tiled products' stage barriers in the compiled code: when a wave reaches the barrier
in front of a stage, its own copies of that stage into LDS must have landed, whatever order
the compiler gave the loads around them (asm_walk)."""
import os

import pytest

from asm_walk import assembly, kernels, unlanded
from tenant_serving_amd import build

pytestmark = pytest.mark.skipif(not os.path.exists(build.HIPCC), reason="no HIP compiler")


@pytest.fixture(scope="module")
def mx4(tmp_path_factory):
    return assembly("bd_mx4.hip", tmp_path_factory.mktemp("asm"))


def test_copies_of_a_stage_land_before_its_barrier(tmp_path):
    """k_gemm: barrier s in front of stage s; bf16 copies W and tokens, INT8 tokens alone."""
    found = kernels(assembly("bd_gemm.hip", tmp_path), "k_gemm")
    assert sum(k[5] for k in found) == 5 and len(found) == 10  # the INT8 and the bf16 tiles
    bad = {}
    for (br, bt, bk, ns, nw, q8), code in found.items():
        per = bt * bk * 2 // 1024 // nw + (0 if q8 else br * bk * 2 // 1024 // nw)
        late = unlanded(code, [s for s in range(20) for _ in range(per)], 9)
        if late:
            bad[f"{br}x{bt}{' int8' if q8 else ''}"] = late
    assert not bad, f"(stage, copies in flight at its barrier): {bad}"


def test_copies_of_the_mx4_token_tiles_land_before_their_barrier(mx4):
    """k_mx4_gemm4: the first period's scales and the copies of NS - 1 stages, then, from
    stage s, the next period's scales (in a period's first stage) and stage s + NS - 1."""
    found = kernels(mx4, "k_mx4_gemm4")
    assert len(found) == 5
    bad = {}
    for (br, bt, kc, ns, nwr, nwt), code in found.items():
        nw, period, rows = nwr * nwt, 512 // kc, 64 // (kc // 32)
        per = br // rows // nw + bt // rows // nw
        scales = ((br + bt + 63) // 64 + nw - 1) // nw
        use = [0] * scales + [s for s in range(ns - 1) for _ in range(per)]
        for s in range(20):
            if s % period == 0:
                use += [s + period] * scales
            use += [s + ns - 1] * per
        late = unlanded(code, use, 12)
        if late:
            bad[f"{br}x{bt}"] = late
    assert not bad, f"(barrier, copies in flight at it): {bad}"


def test_copies_of_the_bf16_token_tiles_land_before_their_barrier(mx4):
    """k_mx4_gemm16: scales of 8 stages, codes of WC / 64 stages and the tokens of one, the
    tokens NSX (WHOLE) or NSX - 1 stages and the codes NSW - 1 slots ahead."""
    found = kernels(mx4, "k_mx4_gemm16")
    assert len(found) == 5
    bad = {}
    for (br, bt, wc, nsx, nsw, nwr, nwt, whole), code in found.items():
        nw, spw = nwr * nwt, wc // 64
        x, w = bt // 8 // nw, br * (wc // 2) // 1024 // nw
        scales = (br // 64 + nw - 1) // nw
        use = [0] * scales
        if whole:  # the prologue in the loop's order
            for t in range(-8, 0):
                if t % spw == 0 and t // spw + nsw - 1 >= 0:
                    use += [(t // spw + nsw - 1) * spw] * w
                if t + nsx >= 0:
                    use += [t + nsx] * x
        else:
            use += [u * spw for u in range(nsw - 1) for _ in range(w)]
            use += [t for t in range(nsx - 1) for _ in range(x)]
        for s in range(20):
            if s % 8 == 0:
                use += [s + 8] * scales
            if s % spw == 0:
                use += [s + (nsw - 1) * spw] * w
            use += [s + nsx - (0 if whole else 1)] * x
        late = unlanded(code, use, 18, 8)
        if late:
            bad[f"{br}x{bt}"] = late
    assert not bad, f"(barrier, copies in flight at it): {bad}"
