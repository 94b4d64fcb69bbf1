"""The layer products', top logits' and distillation's host code under
AddressSanitizer, UndefinedBehaviorSanitizer and LeakSanitizer (no GPU is
used): a C program asks for workspaces from one token to the most, and calls
every entry point with arguments that it refuses."""
import os
import subprocess

import pytest

from tests import sanitize_build as S

PROGRAM = r"""
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include "gradcomp.h"

#define CHECK(c) do { if (!(c)) { printf("FAIL line %d: %s (%s)\n", __LINE__, #c, gc_last_error()); return 1; } } while (0)

int main(void) {
    static const uint32_t shapes[][2] = {{1, 1}, {29, 1600}, {10000, 1500}, {1, 4294967}, {65537, 3}, {16384, 4096}, {127, 129}};
    static const uint64_t tokens[] = {0, 1, 2, 16, 17, 64, 65, 700, 4096, 100000, 1u << 20, (1u << 28) - 1, 1u << 28, ~0ull};
    char *buf = malloc(1 << 16);
    for (size_t i = 0; i < sizeof shapes / sizeof shapes[0]; ++i) {
        const uint32_t rows = shapes[i][0], cols = shapes[i][1];
        gc_segment segs[2] = {{3, rows * cols, 1, 1, 0}, {3 + (uint64_t)rows * cols, rows, 1, 1, 0}};
        gc_plan *p = NULL;
        CHECK(gc_plan_create(segs, 2, segs[1].offset + rows, &p) == GC_OK);
        for (int type = GC_F32; type <= GC_F16; ++type) {
            gc_linear l = {0, rows, 1, type, {0, 0}};
            const uint64_t most = rows > cols ? rows : cols;
            for (size_t t = 0; t < sizeof tokens / sizeof tokens[0]; ++t) {
                const uint64_t n = tokens[t];
                const size_t need = gc_linear_workspace_bytes(p, &l, n);
                const int fits = n < (1u << 28) && n * most <= (1ull << 35);
                CHECK(fits ? need >= 256 && need <= (33u << 20) : need == 0);
                if (!fits || n == 0) continue;
                CHECK(gc_linear_forward(p, &l, buf, buf + 64, cols, n, GC_ACT_GELU, NULL, 0, NULL, 0, buf + 128, rows, buf, need - 1, NULL) == GC_ECAPACITY);
                CHECK(gc_linear_grad_input(p, &l, buf, buf + 64, rows, n, NULL, 0, GC_ACT_NONE, NULL, 0, buf + 128, cols, NULL, 0, buf, need - 1, NULL) == GC_ECAPACITY);
                CHECK(gc_linear_grad_weight(p, &l, buf, rows, buf + 64, cols, n, (float *)(buf + 128), 1, buf, need - 1, NULL) == GC_ECAPACITY);
                CHECK(gc_linear_forward(p, &l, buf, buf + 64, cols, n, 9, NULL, 0, NULL, 0, buf + 128, rows, buf, need, NULL) == GC_EINVAL);
            }
            l.seg = 2;
            CHECK(gc_linear_workspace_bytes(p, &l, 5) == 0);
            l.seg = -1;
            CHECK(gc_linear_workspace_bytes(p, &l, 5) == 0);
            l.seg = 0;
            l.bias_seg = 7;
            CHECK(gc_linear_workspace_bytes(p, &l, 5) == 0);
        }
        gc_plan_destroy(p);
    }
    CHECK(gc_act_grad(buf, 9, buf, 9, GC_ACT_SILU, GC_BF16, 1u << 27, 1u << 20, buf, 9, NULL) == GC_ERANGE);
    CHECK(gc_act_grad(buf, 8, buf, 9, GC_ACT_SILU, GC_BF16, 4, 9, buf, 9, NULL) == GC_EINVAL);
    {
        static const float bad[] = {0.0f, -1.0f, NAN, INFINITY, 1e-40f, 3.2e-39f};
        gc_distill_options o;
        memset(&o, 0, sizeof o);
        o.kd_weight = 1.0f;
        for (size_t i = 0; i < sizeof bad / sizeof bad[0]; ++i) {
            o.temperature = bad[i];
            CHECK(gc_top_logits(buf, GC_F32, 50, 4, 50, 3, bad[i], (int32_t *)buf, (float *)buf, NULL, NULL) == GC_EINVAL);
            CHECK(gc_distill_loss(buf, GC_F32, 50, 4, 50, buf, GC_TOKENS_I32, 3, buf, GC_F32, 3, 3, NULL, NULL, NULL, &o, (float *)buf, NULL, 0, NULL) == GC_EINVAL);
        }
        o.temperature = 3e25f;  /* its square overflows */
        CHECK(gc_distill_loss(buf, GC_F32, 50, 4, 50, buf, GC_TOKENS_I32, 3, buf, GC_F32, 3, 3, NULL, NULL, NULL, &o, (float *)buf, NULL, 0, NULL) == GC_EINVAL);
        o.temperature = 1.0f;
        CHECK(gc_distill_loss(buf, GC_F32, 50, 4, 50, buf, 7, 3, buf, GC_F32, 3, 3, NULL, NULL, NULL, &o, (float *)buf, NULL, 0, NULL) == GC_EINVAL);
        CHECK(gc_distill_loss(buf, GC_F32, 50, 1u << 22, 50, buf, 0, 3, buf, GC_F32, 3, 3, NULL, NULL, NULL, &o, (float *)buf, NULL, 0, NULL) == GC_ERANGE);
        CHECK(gc_distill_loss(buf, GC_F32, 50, 0, 50, NULL, 0, 3, NULL, GC_F32, 3, 3, NULL, NULL, NULL, &o, NULL, NULL, 0, NULL) == GC_OK);
        CHECK(gc_top_logits(buf, GC_F32, 50, 4, GC_MAX_VOCAB + 1, 3, 1.0f, (int32_t *)buf, (float *)buf, NULL, NULL) == GC_ENOTSUP);
    }
    free(buf);
    printf("ok\n");
    return 0;
}
"""


@pytest.mark.skipif(not (os.path.exists(S.CLANG) and os.path.exists(S.hip_build.HIPCC)),
                    reason="needs the ROCm toolchain")
def test_layer_entry_points_under_asan_ubsan_and_lsan(tmp_path):
    out = str(tmp_path)
    S.build_host_library(out)
    src, exe = os.path.join(out, "layers.c"), os.path.join(out, "layers")
    with open(src, "w") as f:
        f.write(PROGRAM)
    r = subprocess.run([S.CLANG, "-std=c99", "-g", "-Wall", "-Werror", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(S.ROOT, "include"), "-I", "/opt/rocm/include", src, "-o", exe,
                        "-L", out, "-lgradcomp", f"-Wl,-rpath,{out}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert r.stdout.strip().endswith("ok")
