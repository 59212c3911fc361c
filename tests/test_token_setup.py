"""Host side of the token operators.  Launches of the products with 4-bit weights over a stand-in for the CUDA runtime,
which keeps a kernel's limits per device as the real one does: what a launch needs is set up on every device it is made
on, once, and a failure is not remembered.  Texts of errors on several threads.  Tensors of another GPU.  Which rows of two tensors meet.  No GPU is needed."""
import os
import subprocess
import types

import pytest
import torch

from rag_kv_cache_rope_gb300 import binding as b
from rag_kv_cache_rope_gb300 import build as B

RUNTIME = r"""
#include <map>
#include <mutex>
#include <utility>
#include "fake.h"
thread_local int device = 0;
int fail_next = 0, launches = 0, sets = 0;
static std::mutex lock;
static std::map<std::pair<int, const void*>, int> limit;
static int enc(void) { return 0; }
static bool fits(const void* f, size_t bytes) {
    std::lock_guard<std::mutex> hold(lock);
    return bytes <= 48 * 1024 || (limit.count({device, f}) && (size_t)limit[{device, f}] >= bytes);
}
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, enum cudaFuncAttribute a, int v) {
    std::lock_guard<std::mutex> hold(lock);
    if (fail_next > 0) { --fail_next; return cudaErrorMemoryAllocation; }
    if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) { limit[{device, f}] = v; ++sets; }
    return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void* f, const cudaLaunchConfig_t* c) {
    if (!fits(f, c->dynamicSmemBytes)) return cudaErrorInvalidValue;
    *n = 152 / (int)c->attrs[0].val.clusterDim.x;
    return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
    if (!fits(f, c->dynamicSmemBytes)) return cudaErrorInvalidValue;
    __atomic_add_fetch(&launches, 1, __ATOMIC_RELAXED);
    return cudaSuccess;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned int, unsigned long long,
                                             enum cudaDriverEntryPointQueryResult* r) {
    *p = (void*)enc;
    *r = cudaDriverEntryPointSuccess;
    return cudaSuccess;
}
void** __cudaRegisterFatBinary(void*) { static void* h; return &h; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, void*, void*, void*, void*, int*) {}
char __cudaInitModule(void**) { return 0; }
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
const char* cudaGetErrorString(cudaError_t) { return "failed"; }
#define NOT_HERE(f) cudaError_t f(void) { return cudaErrorUnknown; }
NOT_HERE(cudaDeviceGetAttribute) NOT_HERE(cudaStreamWaitEvent) NOT_HERE(cudaStreamSynchronize) NOT_HERE(cudaStreamDestroy)
NOT_HERE(cudaStreamCreateWithFlags) NOT_HERE(cudaPointerGetAttributes) NOT_HERE(cudaMemsetAsync) NOT_HERE(cudaMemcpyAsync)
NOT_HERE(cudaGetSymbolAddress) NOT_HERE(cudaGetDeviceProperties) NOT_HERE(cudaEventSynchronize) NOT_HERE(cudaEventRecord)
NOT_HERE(cudaEventElapsedTime) NOT_HERE(cudaEventDestroy) NOT_HERE(cudaEventCreateWithFlags) NOT_HERE(cudaEventCreate)
unsigned __cudaPushCallConfiguration(void) { return 1; }
cudaError_t __cudaPopCallConfiguration(void) { return cudaErrorUnknown; }
cudaError_t __cudaGetKernel(void) { return cudaErrorUnknown; }
cudaError_t __cudaLaunchKernel(void) { return cudaErrorUnknown; }
}
"""

FAKE_H = r"""
#pragma once
#include <driver_types.h>
#include <stddef.h>
extern thread_local int device;
extern int fail_next, launches, sets;
"""

CALLS = r"""
#include <stdio.h>
#include <thread>
#include <vector>
#include "tokens.cuh"
#include "fake.h"
namespace blend {
void note_launch(int) {}
}
using namespace blend;
static int call(int rows, int group, int dtype = BLEND_BF16) {
    static char mem[64] __attribute__((aligned(64)));
    W4Linear a = {};
    a.w.codes = (const uint4*)mem;
    a.w.scale = (const bf16*)mem;
    a.w.n = 5120;
    a.w.k = 8192;
    a.w.group = group;
    a.w.chunks = 64;
    a.x = a.y = mem;
    a.ld_x = 8192;
    a.ld_y = 5120;
    a.rows = rows;
    a.y_f32 = 1;
    a.tc = true;
    return launch_w4_linear(dtype, a, 0);
}
#define WANT(x) do { if (!(x)) { printf("%d: " #x "\n", __LINE__); return 1; } } while (0)
int main(void) {
    for (int d = 0; d < 3; ++d) {
        device = d;
        for (int rows : {1, 8, 30, 60, 500}) {
            WANT(call(rows, 128) == BLEND_OK);
            const int before = sets;
            WANT(call(rows, 128) == BLEND_OK && sets == before);
        }
        WANT(call(3, 128, BLEND_F32) == BLEND_OK);
    }
    WANT(launches == 3 * 11);
    // a failure is that call's alone
    for (int rows : {2, 500}) {
        device = 1;
        fail_next = 1;
        WANT(call(rows, 64) == BLEND_ECUDA);
        WANT(call(rows, 64) == BLEND_OK);
    }
    // first calls of several threads on several devices at once
    std::vector<std::thread> t;
    int bad[8] = {};
    for (int i = 0; i < 8; ++i)
        t.emplace_back([&bad, i] {
            device = i % 4;
            for (int rows : {1, 30, 60, 500}) bad[i] += call(rows, 32) != BLEND_OK;
        });
    for (auto& x : t) x.join();
    for (int b : bad) WANT(b == 0);
    return 0;
}
"""


def run_over_stand_in(tmp_path, name, source, objects):
    """Builds `source` with the library's objects and the stand-in for the CUDA runtime, and runs it."""
    B.build()
    (tmp_path / "fake.h").write_text(FAKE_H)
    (tmp_path / "runtime.cpp").write_text(RUNTIME)
    (tmp_path / name).write_text(source)
    inc = ["-I", str(tmp_path), "-I", B.CSRC, "-I", os.path.join(B.ROOT, "include"),
           "-I", os.path.join(os.path.dirname(os.path.dirname(B.nvcc())), "include")]
    objs = []
    for f in ("runtime.cpp", name):
        cc = ["g++"] if f.endswith(".cpp") else [B.nvcc(), *B.ARCH]
        objs.append(str(tmp_path / (f + ".o")))
        subprocess.run([*cc, "-std=c++17", *inc, "-c", str(tmp_path / f), "-o", objs[-1]], check=True)
    exe = str(tmp_path / "probe")
    subprocess.run(["g++", *objs, *objects, "-o", exe, "-lpthread", "-ldl"], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, (r.returncode, r.stdout + r.stderr)


def test_launches_on_every_device_and_after_a_failure(tmp_path):
    run_over_stand_in(tmp_path, "calls.cu", CALLS, [os.path.join(B.BUILD, f + ".cu.o") for f in ("w4", "w4_tile")])


ERRORS = r"""
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <string>
#include <thread>
#include <vector>
#include "blend.h"
int main(void) {
    blend_model_cfg cfg = {1, 16, 4, 2, 128, 16, 16, BLEND_BF16, 1e4, 1e-6, 64};
    blend_limits lim = {1, 1, 1, 1};
    const size_t bytes = blend_workspace_size(&cfg, &lim);
    void* ws = aligned_alloc(256, (bytes + 255) / 256 * 256);
    static char mem[4096] __attribute__((aligned(256)));
    blend_weights w = {mem, mem, mem, mem, mem, mem, mem, mem};
    blend_handle *h = nullptr, *other = nullptr;
    if (blend_init(&cfg, &w, &lim, ws, bytes, nullptr, &h) || blend_init(&cfg, &w, &lim, ws, bytes, nullptr, &other)) {
        printf("no handle: %s\n", blend_last_error(nullptr));
        return 1;
    }
    int wrong[4] = {};
    std::vector<std::thread> t;
    for (int i = 0; i < 4; ++i)
        t.emplace_back([&, i] {
            for (int n = 0; n < 20000; ++n) {
                blend_w4 w4 = {32, 128, 48 + 1000 * i + n, mem, mem};
                char want[64];
                int rc;
                if (i % 2) {
                    rc = w4_linear(h, &w4, mem, 128, 1, mem, 32, BLEND_F32, BLEND_W4_STORE, nullptr);
                    snprintf(want, sizeof want, "group=%d is not 32, 64 or 128", w4.group);
                } else {
                    rc = token_logprobs(h, i ? mem : nullptr, 1, 5 + n, 1, 1, 1.f, nullptr, 0, nullptr, nullptr, 0, nullptr, nullptr, nullptr);
                    if (i) snprintf(want, sizeof want, "bad dtype %d", 5 + n);
                    else snprintf(want, sizeof want, "NULL pointer");
                }
                wrong[i] += rc != BLEND_EINVAL || strcmp(blend_last_error(h), want) || strcmp(blend_last_error(nullptr), want);
            }
        });
    for (auto& x : t) x.join();
    for (int i = 0; i < 4; ++i)
        if (wrong[i]) {
            printf("thread %d: %d texts of other calls\n", i, wrong[i]);
            return 2;
        }
    // one thread, two handles; another thread's text; a handle that follows one
    w4_unpack(h, nullptr, mem, 8, nullptr);
    w4_unpack(other, nullptr, nullptr, 8, nullptr);
    rope_rows(other, nullptr, nullptr, 1, nullptr, nullptr, 1, nullptr);
    if (strcmp(blend_last_error(h), "w4 is NULL") || strcmp(blend_last_error(other), "NULL pointer")) return 3;
    std::thread([&] { token_logprobs(h, mem, 1, 7, 1, 1, 1.f, nullptr, 0, nullptr, nullptr, 0, nullptr, nullptr, nullptr); }).join();
    if (strcmp(blend_last_error(h), "bad dtype 7")) return 4;
    std::string seen;
    std::thread([&] { seen = blend_last_error(h); }).join();
    return seen == "bad dtype 7" ? 0 : 5;
}
"""


def test_texts_of_calls_that_fail_on_several_threads(tmp_path):
    """Refused calls of one handle on four threads: each reads its own text (and none another's half written)."""
    run_over_stand_in(tmp_path, "errors.cpp", ERRORS, [os.path.join(B.BUILD, os.path.basename(f) + ".o") for f in B._sources()])


class Tensor(torch.Tensor):
    """A tensor that says that it is on the second GPU."""

    def get_device(self):
        return 1


def test_tensors_on_another_gpu_than_the_handle_are_refused(monkeypatch):
    """A handle's error word lies on its own GPU, so a kernel on another must not get it."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 0, raising=False)
    h = types.SimpleNamespace(ptr=None, index=0, cfg=types.SimpleNamespace(dtype=b.BF16, head_dim=128, n_kv_heads=2, n_q_heads=4))

    def at(t):
        return t.as_subclass(Tensor)

    w4 = b.W4Ref(at(torch.zeros(32, 64, dtype=torch.uint8)), torch.zeros(32, 1, dtype=torch.bfloat16), 128)
    x, y = at(torch.zeros(1, 128, dtype=torch.bfloat16)), at(torch.zeros(1, 32))
    k, one = at(torch.zeros(1, 2, 128, dtype=torch.bfloat16)), at(torch.ones(1, dtype=torch.int32))
    w = at(torch.zeros(32, 128, dtype=torch.bfloat16))
    for call in (lambda: b.w4_linear(h, w4, x, y), lambda: b.w4_pack(h, w, w4), lambda: b.w4_unpack(h, w4, w),
                 lambda: b.token_logprobs(h, y, entropy=at(torch.zeros(1))),
                 lambda: b.rope_rows(h, b.rope_desc(1e4, 128), k, k, one, one, 1)):
        with pytest.raises(ValueError, match="the handle on cuda:0"):
            call()


MEET = r"""
#include <stdio.h>
#include <stdlib.h>
#include "tokens.cuh"
static long long r(long long lo, long long hi) { return lo + rand() % (hi - lo + 1); }
int main(void) {
    srand(7);
    static char a[4096], b[4096];
    long long met = 0, apart = 0, wide = 0;
    for (int t = 0; t < 400000; ++t) {
        const long long n = r(1, 5), wa = r(1, 9), wb = r(1, 9), la = r(1, 4), lb = r(1, 4);
        const bool alike = t % 8 != 0;
        long long row_a = r(9, 40), row_b = alike ? row_a : r(9, 40);
        long long layer_a = r(9, 120), layer_b = alike ? layer_a : r(9, 120);
        if (n == 1 && t % 2) row_b = r(9, 40);       // a step that is not taken
        if (la == 1 && t % 3) layer_a = r(0, 400) - 200;
        if (lb == 1 && t % 3 == 1) layer_b = r(0, 400) - 200;
        const long long pa = r(0, 300), pb = r(0, 300);
        bool want = false;
        for (long long l = 0; l < la; ++l)
            for (long long i = 0; i < n; ++i)
                for (long long m = 0; m < lb; ++m)
                    for (long long j = 0; j < n; ++j) {
                        const long long x = pa + (la > 1 ? l * layer_a : 0) + i * row_a, y = pb + (lb > 1 ? m * layer_b : 0) + j * row_b;
                        want |= x < y + wb && y < x + wa;
                    }
        const bool got = blend::rows_meet(a + pa, row_a, layer_a, la, wa, a + pb, row_b, layer_b, lb, wb, n);
        const bool steps = (n == 1 || row_a == row_b) && (la == 1 || lb == 1 || layer_a == layer_b);
        if (steps ? got != want : want && !got) {
            printf("n %lld rows %lld %lld layers %lld x %lld, %lld x %lld at %lld %lld: %d\n", n, row_a, row_b, la, layer_a, lb, layer_b, pa, pb, got);
            return 1;
        }
        bool in = false;  // b's first row alone
        for (long long l = 0; l < la; ++l)
            for (long long i = 0; i < n; ++i) {
                const long long x = pa + (la > 1 ? l * layer_a : 0) + i * row_a;
                in |= x < pb + wb && pb < x + wa;
            }
        if (blend::bytes_meet_rows(b + pb, wb, b + pa, row_a, layer_a, la, wa, n) != in) {
            printf("%lld bytes at %lld, n %lld row %lld layers %lld x %lld width %lld at %lld: %d\\n", wb, pb, n, row_a, la, layer_a, wa, pa, !in);
            return 5;
        }
        met += want;
        apart += !want && steps;
        wide += got && !want;
    }
    // many layers of long rows, far apart in one buffer, and the same layers
    char* p = 0;
    const long long row = 3ll << 20, layer = row << 18;
    if (blend::rows_meet(p, row, layer, 1 << 16, 4096, p + 4096, row, layer, 1 << 16, 4096, 1 << 18)) return 2;
    if (!blend::rows_meet(p, row, layer, 1 << 16, 4096, p + 4080, row, layer, 1 << 16, 4096, 1 << 18)) return 3;
    printf("%lld %lld %lld\n", met, apart, wide);
    return met > 1000 && apart > 1000 && (b[0] == 0) ? 0 : 4;
}
"""


def test_which_rows_meet(tmp_path):
    """Against every pair of rows, for small tensors of any steps."""
    src, exe = tmp_path / "probe.cu", tmp_path / "probe"
    src.write_text(MEET)
    subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "-I", B.CSRC, "-I", os.path.join(B.ROOT, "include"), str(src), "-o", str(exe)],
                   check=True, capture_output=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stdout)
