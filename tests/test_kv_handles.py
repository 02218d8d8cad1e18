"""What the key-value cache's and the block norm's calls ask the HIP runtime (csrc/kv.cpp) over a stand-in for it with
two devices: a stream of another device than the current one is refused, handles that are no stream objects are not asked
about, and a call without rows launches nothing.  A small harness includes the sources, compiled as the library compiles
them.  CPU only."""
import os
import subprocess

from moe_expert_execution_amd.build import HIPCC

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
COMPILER = os.path.join(os.path.dirname(HIPCC), "amdclang++")
PKG = os.path.join(ROOT, "moe_expert_execution_amd", "csrc")

RESIDENT = '#include "resident.cpp"\n'
HARNESS = r"""
#include <stdarg.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include "kv.cpp"

static int current = 0, stream_device = 0, calls = 0;
extern "C" {
hipError_t hipGetDevice(int* d) { *d = current; return hipSuccess; }
hipError_t hipSetDevice(int d) { current = d; return hipSuccess; }
hipError_t hipMalloc(void** p, size_t n) { *p = malloc(64); return hipSuccess; }
hipError_t hipFree(void* p) { free(p); return hipSuccess; }
hipError_t hipMemset(void*, int, size_t) { return hipSuccess; }
hipError_t hipDeviceSynchronize() { return hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "error"; }
hipError_t hipStreamGetDevice(hipStream_t s, hipDevice_t* d) {
    if ((uintptr_t)s <= 2) { printf("the runtime was asked for a special stream\n"); exit(9); }
    *d = stream_device;
    return hipSuccess;
}
}
namespace ftmoe {
char err[512];
void set_error(const char* f, ...) { va_list a; va_start(a, f); vsnprintf(err, sizeof(err), f, a); va_end(a); }
void clear_error() { err[0] = 0; }
bool record_layout(const ft_shape&, RecordLayout* o) { memset(o, 0, sizeof(*o)); return true; }
hipError_t launch_layer(const ft_shape&, const LayerArgs&, ft_workspace*, hipStream_t) { return hipSuccess; }
hipError_t launch_lora_project(const MatrixView&, const LoraView*, const int32_t*, const uint16_t*, int, const uint16_t*,
                               uint16_t*, ft_workspace*, hipStream_t) { return hipSuccess; }
hipError_t launch_lora_expert(const ft_shape&, const RecordLayout&, const uint8_t*, const LoraView*, const LoraView*,
                              const LoraView*, const int32_t*, const uint16_t*, int, const uint16_t*, uint16_t*,
                              ft_workspace*, hipStream_t) { return hipSuccess; }
size_t layer_call_bytes(const ft_shape&, int) { return 0; }
size_t layer_workspace(const ft_shape&, int) { return 0; }
size_t lora_project_call_bytes(int, int, int, int) { return 0; }
size_t lora_expert_call_bytes(const ft_shape&, int, int) { return 0; }
size_t lora_project_workspace(int, int, int, int) { return 0; }
size_t lora_expert_workspace(const ft_shape&, int, int) { return 0; }
hipError_t launch_kv_plan(const ft_kv_batch&, ft_workspace*, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_kv_append(const CacheView&, const ft_append&, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_kv_attend(const CacheView&, const ft_attend&, ft_workspace*, hipStream_t) { ++calls; return hipSuccess; }
size_t kv_attend_workspace(int, int) { return 64; }
hipError_t launch_block_norm(const ft_norm&, hipStream_t) { ++calls; return hipSuccess; }
}
#define CHECK(c) do { if (!(c)) { printf("line %d: %s (%s)\n", __LINE__, #c, ftmoe::err); return 1; } } while (0)

int main() {
    alignas(64) static char mem[256];
    int32_t* i = (int32_t*)mem;
    uint16_t *u = (uint16_t*)mem, *v = (uint16_t*)(mem + 128);
    ft_kv_cache c = {4, 16, 1, 64, FT_KV_BF16, 0, 2048, mem, mem, nullptr, nullptr};
    ft_append a = {2, 0, 0, 0, nullptr, u, u, 0, 64, 64, i, nullptr, nullptr, nullptr, 0};
    ft_attend t = {2, 1, 3, 0, 1.0f, 0, u, 64, i, i, nullptr, v, 64};
    ft_kv_batch b = {2, 4, 16, 3, 2, 1, i, i, i, i, i, i, i, i, i, i};
    ft_norm n = {2, 64, 0, 1e-6f, 1.0f, 0.0f, u, nullptr, nullptr, nullptr, nullptr, v, nullptr, 64, 64, 64, 64, 64};
    ft_workspace* ws = nullptr;
    CHECK(ft_workspace_create(64, &ws) == FT_OK);
    void* created = mem;
    auto all = [&](void* s, ft_status want, const char* words) {
        const ft_status got[] = {ft_kv_plan(&b, ws, s), ft_kv_append(&c, &a, s), ft_kv_attend(&c, &t, ws, s), ft_block_norm(&n, s)};
        for (ft_status g : got) if (g != want) return false;
        return want == FT_OK || strstr(ftmoe::err, words) != nullptr;
    };
    CHECK(all(nullptr, FT_OK, "") && calls == 4);
    CHECK(all(created, FT_OK, "") && calls == 8);
    CHECK(all((void*)hipStreamLegacy, FT_ERR_ARG, "hipStreamLegacy") && all((void*)hipStreamPerThread, FT_ERR_ARG, "hipStreamPerThread"));
    stream_device = 1;                                // the stream of another device than the current one
    CHECK(all(created, FT_ERR_ARG, "belongs to device 1") && calls == 8);
    current = 1;                                      // both on another device than the workspace
    CHECK(ft_kv_append(&c, &a, created) == FT_OK && ft_block_norm(&n, created) == FT_OK && calls == 10);
    CHECK(ft_kv_plan(&b, ws, created) == FT_ERR_ARG && ft_kv_attend(&c, &t, ws, created) == FT_ERR_ARG);
    CHECK(ft_kv_plan(&b, ws, nullptr) == FT_ERR_ARG && strstr(ftmoe::err, "device 1 is current"));
    current = stream_device = 0;
    ft_workspace* small = nullptr;
    CHECK(ft_workspace_create(63, &small) == FT_OK);
    CHECK(ft_kv_attend(&c, &t, small, nullptr) == FT_ERR_ARG && ft_kv_plan(&b, small, nullptr) == FT_OK && calls == 11);
    CHECK(ft_workspace_destroy(small) == FT_OK);
    CHECK(ft_kv_plan(&b, small, nullptr) == FT_ERR_ARG && strstr(ftmoe::err, "not a workspace"));
    a.tokens = 0, t.requests = 0, b.requests = 0, b.tokens = 0, n.T = 0;
    CHECK(all(nullptr, FT_OK, "") && calls == 11);
    CHECK(ft_workspace_destroy(ws) == FT_OK);
    printf("ok\n");
    return 0;
}
"""


def test_what_the_runtime_is_asked(tmp_path):
    (tmp_path / "kv_main.cpp").write_text(HARNESS)
    (tmp_path / "resident_part.cpp").write_text(RESIDENT)
    exe = tmp_path / "h"
    flags = ["-x", "c++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", PKG,
             "-I", "/opt/rocm/include", "-Wno-c++20-extensions", "-Wno-unused-value", "-Wno-deprecated-declarations"]
    subprocess.check_call([COMPILER] + flags + [str(tmp_path / "kv_main.cpp"), str(tmp_path / "resident_part.cpp"), "-o",
                                                str(exe), "-pthread"])
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.stdout == "ok\n", r.stdout + r.stderr
