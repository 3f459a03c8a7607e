"""How many CTAs of the norms' kernels stand on an SM: what is asked for has to fit, or the last of them run as a second
wave.  The launch's own arithmetic, compiled for the host."""
import os
import subprocess

from sparse_expert_ffn_route_gb300 import build

PROGRAM = r"""
#include <cstdio>
#include "block_norm.cuh"
using namespace moe;
using namespace moe::norm;
// 228 KB an SM, of which each CTA takes its own, in pieces of 128 bytes, and 1 KB of the system's; 32 CTAs at most
bool fits(int ctas, int bytes) { return ctas <= 32 && ctas * ((bytes + 127) / 128 * 128 + 1024) <= 228 * 1024; }
int main()
{
    int bad = 0, seen = 0;
    char operand;
    for (int H = 8; H <= kMaxDim; H += 8)
        for (int ex : {2, 4})
            for (int ey : {2, 4})
                for (int what = 0; what < 16; ++what) {   // dout, y, dn and a full gate, each there or not
                    NormArgs p = {};
                    p.H = H;
                    p.dout = what & 1 ? &operand : nullptr;
                    p.y = what & 2 ? &operand : nullptr;
                    p.dn = what & 4 ? &operand : nullptr;
                    p.kind = what & 8 ? kGateFull : kGateNone;
                    const int row = (int)RowBytes(p, ex, ey).total();
                    for (int T : {1, 100, 304, 305, 2000, 5000, 100000, 1 << 24})
                        for (int heavy = 0; heavy < 3; ++heavy) {
                            const int parts = norm_parts(T, H, heavy), most = ctas_per_sm(H, heavy);
                            const int stages = backward_stages(row, parts, most);
                            const int there = (parts + 151) / 152;
                            ++seen;
                            if (stages < 1 || stages > kMaxNormStages || there > most || !fits(there, stages * row + (int)sizeof(BackwardShared)))
                                if (bad++ < 20) printf("backward: H %d, a row of %d bytes: %d CTAs of %d stages\n", H, row, there, stages);
                        }
                    const int ring = kRowStages * H * (ex + (p.y ? ey : 0) + (p.kind == kGateFull ? ey : 0));
                    const int threads = norm_threads(H, kVecs), fit = forward_ctas(threads, ring);
                    ++seen;
                    if (fit > 1 && !fits(fit, ring + (int)sizeof(RowsShared)))
                        if (bad++ < 20) printf("forward: H %d, a ring of %d bytes: %d CTAs\n", H, ring, fit);
                }
    printf("%d of %d do not fit\n", bad, seen);
    return bad != 0;
}
"""


def test_the_ctas_fit_the_sm(tmp_path):
    source, program = tmp_path / "plan.cu", tmp_path / "plan"
    source.write_text(PROGRAM)
    flags = [f for f in build.NVCC_FLAGS if f != "-lineinfo"]
    r = subprocess.run([build.nvcc(), *build.ARCH, *flags, str(source), "-o", str(program)], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(program)], capture_output=True, text=True, env={**os.environ, "CUDA_VISIBLE_DEVICES": ""}, timeout=120)
    assert r.returncode == 0, r.stdout
