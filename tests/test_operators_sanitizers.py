"""The embedding and matrix-plan entry points' host code under AddressSanitizer,
UndefinedBehaviorSanitizer and LeakSanitizer (no GPU is used): a C program
makes and destroys plans of many shapes, which plans their work lists, and
calls every entry point with arguments that it refuses."""
import os
import subprocess

import pytest

from tests import sanitize_build as S

PROGRAM = r"""
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include "gradcomp.h"

#define CHECK(c) do { if (!(c)) { printf("FAIL line %d: %s (%s)\n", __LINE__, #c, gc_last_error()); return 1; } } while (0)

static gc_matrix_plan *plan_of(const uint32_t (*shape)[2], int n) {
    gc_segment *segs = calloc((size_t)n, sizeof *segs);
    uint32_t *rows = calloc((size_t)n, sizeof *rows);
    gc_plan *p = NULL;
    gc_matrix_plan *m = NULL;
    uint64_t at = 0;
    int i;
    for (i = 0; i < n; ++i) {
        segs[i].offset = at;
        segs[i].length = shape[i][0] * shape[i][1];
        segs[i].bin_len = 1;
        segs[i].k = 1;
        rows[i] = shape[i][0];
        at += segs[i].length;
    }
    if (gc_plan_create(segs, n, at, &p) == GC_OK && gc_matrix_plan_create(p, rows, &m) != GC_OK) m = NULL;
    gc_plan_destroy(p);
    free(segs);
    free(rows);
    return m;
}

int main(void) {
    static const uint32_t shapes[][2] = {{1, 1}, {29, 1600}, {1600, 29}, {128, 5000}, {129, 5000}, {1500, 6000}, {4096, 4096},
                                         {1, 1000000}, {65000, 300}, {2400, 8640}, {300, 70}};
    const int n = (int)(sizeof shapes / sizeof shapes[0]);
    void *buf = malloc(4096);
    int i;
    for (i = 0; i < n; ++i) {
        gc_matrix_plan *m = plan_of(shapes + i, 1);
        gc_orth_options o;
        CHECK(m != NULL && gc_matrix_plan_workspace_bytes(m) > 0);
        memset(&o, 0, sizeof o);
        CHECK(gc_orthogonalize(m, buf, buf, &o, buf, 4096, NULL) == GC_EINVAL);
        o.steps = GC_MAX_ORTH_STEPS;
        for (int k = 0; k < o.steps; ++k) { o.coef[k][0] = 3.4445f; o.coef[k][1] = -4.775f; o.coef[k][2] = 2.0315f; }
        CHECK(gc_orthogonalize(m, buf, buf, &o, buf, 16, NULL) == GC_ECAPACITY);
        gc_matrix_plan_destroy(m);
    }
    {
        gc_matrix_plan *m = plan_of(shapes, n);  /* all of them in one plan */
        CHECK(m != NULL);
        gc_matrix_plan_destroy(m);
    }
    {
        gc_segment seg = {3, 120, 1, 1, 0};
        gc_plan *p = NULL;
        gc_sparse msg;
        memset(&msg, 0, sizeof msg);
        CHECK(gc_plan_create(&seg, 1, 200, &p) == GC_OK);
        CHECK(gc_embed_workspace_bytes(p, 0, 10, 5) > 0 && gc_embed_message_cap(p, 0, 10, 5) == 60);
        CHECK(gc_embed_lookup(p, 0, 10, buf, buf, GC_TOKENS_I32, 0, 1.0f, buf, GC_F32, 12, NULL) == GC_OK);
        CHECK(gc_embed_lookup(p, 0, 7, buf, buf, GC_TOKENS_I32, 1, 1.0f, buf, GC_F32, 12, NULL) == GC_EINVAL);
        CHECK(gc_embed_grad(p, 0, 10, buf, GC_BF16, 12, buf, GC_TOKENS_I64, 5, 1.0f, buf, 0, buf, 8, NULL) == GC_ECAPACITY);
        CHECK(gc_embed_message(p, 0, 10, buf, GC_F16, 12, buf, GC_TOKENS_I64, 5, 1.0f, &msg, buf, 8, NULL) == GC_EINVAL);
        gc_plan_destroy(p);
    }
    free(buf);
    printf("ok\n");
    return 0;
}
"""


@pytest.mark.skipif(not (os.path.exists(S.CLANG) and os.path.exists(S.hip_build.HIPCC)),
                    reason="needs the ROCm toolchain")
def test_operator_entry_points_under_asan_ubsan_and_lsan(tmp_path):
    out = str(tmp_path)
    S.build_host_library(out)
    src, exe = os.path.join(out, "operators.c"), os.path.join(out, "operators")
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


SCHEDULES = r"""
#include <math.h>
#include <stdio.h>
#include <string.h>
#include "gradcomp.h"

/* Coefficients that are not finite, overflow, or let X vanish: each is an
   error, and none a number that an int cannot hold on the way there. */
int main(void) {
    static const float coef[][3] = {{0, 0, 0}, {NAN, 0, 0}, {1, NAN, 0}, {1, 0, NAN}, {1, 0, INFINITY}, {-INFINITY, INFINITY, 0},
                                    {3e38f, 3e38f, 3e38f}, {-3e38f, 3e38f, 0}, {1e-30f, 0, 0}, {0, 1e-38f, 0}, {0, 0, 1e-45f}};
    static float buf[4096];
    gc_segment seg = {0, 120, 1, 1, 0};
    uint32_t rows = 10;
    gc_plan *p = NULL;
    gc_matrix_plan *m = NULL;
    if (gc_plan_create(&seg, 1, 120, &p) != GC_OK || gc_matrix_plan_create(p, &rows, &m) != GC_OK) return 1;
    for (unsigned i = 0; i < sizeof coef / sizeof coef[0]; ++i)
        for (int at = 0; at < GC_MAX_ORTH_STEPS; ++at)
            for (int steps = at + 1; steps <= GC_MAX_ORTH_STEPS; steps += 5) {
                gc_orth_options o;
                memset(&o, 0, sizeof o);
                o.steps = steps;
                for (int k = 0; k < steps; ++k) { o.coef[k][0] = 1.5f; o.coef[k][1] = -0.5f; }
                memcpy(o.coef[at], coef[i], sizeof coef[i]);
                if (gc_orthogonalize(m, buf, buf, &o, buf, 16, NULL) != GC_EINVAL) {
                    printf("coefficients %u in step %d of %d\n", i, at, steps);
                    return 1;
                }
            }
    gc_matrix_plan_destroy(m);
    gc_plan_destroy(p);
    printf("ok\n");
    return 0;
}
"""


@pytest.mark.skipif(not (os.path.exists(S.CLANG) and os.path.exists(S.hip_build.HIPCC)),
                    reason="needs the ROCm toolchain")
def test_refused_schedules_under_asan_and_ubsan(tmp_path):
    out = str(tmp_path)
    S.build_host_library(out)
    src, exe = os.path.join(out, "schedules.c"), os.path.join(out, "schedules")
    with open(src, "w") as f:
        f.write(SCHEDULES)
    r = subprocess.run([S.CLANG, "-std=c99", "-g", "-Wall", "-Werror", "-fsanitize=address,undefined",
                        "-fno-sanitize-recover=all", "-fno-omit-frame-pointer", "-D__HIP_PLATFORM_AMD__",
                        "-I", os.path.join(S.ROOT, "include"), "-I", "/opt/rocm/include", src, "-o", exe,
                        "-L", out, "-lgradcomp", f"-Wl,-rpath,{out}"], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=1:halt_on_error=1", UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, r.stdout[-4000:] + r.stderr[-4000:]
    assert r.stdout.strip().endswith("ok")
