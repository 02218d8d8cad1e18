"""The workspace handle (csrc/resident.cpp) over a stand-in for the HIP runtime with two devices: destroying waits for
and frees on the workspace's own device, leaves the current one as it was, and never reads a destroyed handle; the
runtime is not asked about handles that are no stream objects.  A small harness includes the source, compiled as the
library compiles it.  CPU only."""
import os
import subprocess

import pytest

from moe_expert_execution_amd.build import HIPCC

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
COMPILER = os.path.join(os.path.dirname(HIPCC), "amdclang++")
PKG = os.path.join(ROOT, "moe_expert_execution_amd", "csrc")

HARNESS = r"""
#include <stdarg.h>
#include <sys/mman.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>
#include <new>
#include "resident.cpp"

// a freed object's page cannot be read any more
void* operator new(size_t n, const std::nothrow_t&) noexcept {
    void* p = mmap(nullptr, 4096, PROT_READ | PROT_WRITE, MAP_PRIVATE | MAP_ANONYMOUS, -1, 0);
    return n <= 4096 && p != MAP_FAILED ? p : nullptr;
}
void operator delete(void* p) noexcept { if (p) mprotect(p, 4096, PROT_NONE); }
void operator delete(void* p, size_t) noexcept { if (p) mprotect(p, 4096, PROT_NONE); }

static int current = 0, synced = -1, freed_on = -1, stream_device = 0, busy = 0;
extern "C" {
hipError_t hipGetDevice(int* d) { *d = current; return hipSuccess; }
hipError_t hipSetDevice(int d) { current = d; return d >= 0 && d < 2 ? hipSuccess : hipErrorInvalidDevice; }
hipError_t hipMalloc(void** p, size_t n) { *p = malloc(64); return hipSuccess; }
hipError_t hipFree(void* p) { freed_on = current; free(p); return hipSuccess; }
hipError_t hipMemset(void*, int, size_t) { return hipSuccess; }
hipError_t hipDeviceSynchronize() { synced = current; return busy ? hipErrorStreamCaptureUnsupported : hipSuccess; }
hipError_t hipGetLastError() { return hipSuccess; }
const char* hipGetErrorString(hipError_t) { return "error"; }
hipError_t hipStreamGetDevice(hipStream_t s, hipDevice_t* d) {
    if ((uintptr_t)s <= 2) { printf("the runtime was asked for a special stream\n"); exit(9); }
    *d = stream_device;
    return hipSuccess;
}
}
namespace ftmoe {
static char err[512];
void set_error(const char* f, ...) { va_list a; va_start(a, f); vsnprintf(err, sizeof(err), f, a); va_end(a); }
void clear_error() { err[0] = 0; }
bool record_layout(const ft_shape&, RecordLayout* o) { memset(o, 0, sizeof(*o)); return true; }
static int calls = 0;
hipError_t launch_layer(const ft_shape&, const LayerArgs&, ft_workspace*, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_lora_project(const MatrixView&, const LoraView*, const int32_t*, const uint16_t*, int, const uint16_t*,
                               uint16_t*, ft_workspace*, hipStream_t) { ++calls; return hipSuccess; }
hipError_t launch_lora_expert(const ft_shape&, const RecordLayout&, const uint8_t*, const LoraView*, const LoraView*,
                              const LoraView*, const int32_t*, const uint16_t*, int, const uint16_t*, uint16_t*,
                              ft_workspace*, hipStream_t) { ++calls; return hipSuccess; }
size_t layer_call_bytes(const ft_shape&, int) { return 1; }
size_t layer_workspace(const ft_shape&, int) { return 1; }
size_t lora_project_call_bytes(int, int, int, int) { return 1; }
size_t lora_expert_call_bytes(const ft_shape&, int, int) { return 1; }
size_t lora_project_workspace(int, int, int, int) { return 1; }
size_t lora_expert_workspace(const ft_shape&, int, int) { return 1; }
}

static int layer(ft_workspace* ws, void* stream) {
    ft_shape s = {};
    s.layers = 1; s.experts = 8; s.top_k = 2; s.d_model = 256; s.d_ff = 128;
    uint16_t* p = (uint16_t*)64;
    return ft_moe_layer(&s, p, p, p, 4096, 1, nullptr, (int32_t*)64, (float*)64, p, ws, stream);
}
static int project(ft_workspace* ws, void* stream) {
    ft_matrix m = {256, 256, FT_FMT_BF16, 0, (void*)64, nullptr};
    return ft_lora_project(&m, nullptr, (uint16_t*)64, nullptr, 1, nullptr, (uint16_t*)64, ws, stream);
}
static int expert(ft_workspace* ws, void* stream) {
    ft_shape s = {};
    s.layers = 1; s.experts = 8; s.top_k = 2; s.d_model = 256; s.d_ff = 128;
    return ft_lora_expert(&s, (void*)64, nullptr, nullptr, nullptr, (uint16_t*)64, nullptr, 1, nullptr, (uint16_t*)64, ws, stream);
}
#define CHECK(c) do { if (!(c)) { printf("line %d: %s (%s)\n", __LINE__, #c, ftmoe::err); exit(1); } } while (0)

int main(int argc, char** argv) {
    const char* what = argv[1];
    ft_workspace *a, *b;
    current = 1;
    CHECK(ft_workspace_create(100, &a) == FT_OK);
    CHECK(ft_workspace_create(100, &b) == FT_OK);
    if (!strcmp(what, "device")) {
        current = 0;
        synced = freed_on = -1;
        CHECK(ft_workspace_destroy(a) == FT_OK);
        CHECK(synced == 1 && freed_on == 1 && current == 0);
        CHECK(layer(b, nullptr) == FT_ERR_ARG && strstr(ftmoe::err, "device 0 is current"));
        current = 1;
        CHECK(layer(b, nullptr) == FT_OK && layer(b, (void*)4096) == FT_ERR_ARG);   // (a stream of device 0)
        stream_device = 1;
        CHECK(layer(b, (void*)4096) == FT_OK && project(b, (void*)4096) == FT_OK && expert(b, nullptr) == FT_OK);
        CHECK(ftmoe::calls == 4);
    } else if (!strcmp(what, "destroyed")) {
        CHECK(ft_workspace_destroy(a) == FT_OK);
        CHECK(ft_workspace_destroy(a) == FT_ERR_ARG && strstr(ftmoe::err, "destroyed"));
        CHECK(layer(a, nullptr) == FT_ERR_ARG && project(a, nullptr) == FT_ERR_ARG && expert(a, nullptr) == FT_ERR_ARG);
        CHECK(layer(b, nullptr) == FT_OK);
        CHECK(ft_workspace_destroy(b) == FT_OK && ft_workspace_destroy(nullptr) == FT_OK);
        CHECK(layer(b, nullptr) == FT_ERR_ARG && ftmoe::calls == 1);
    } else if (!strcmp(what, "capturing")) {      // a wait that the runtime refuses: nothing is freed, and it may be tried again
        current = 0;
        busy = 1;
        CHECK(ft_workspace_destroy(a) == FT_ERR_HIP && freed_on == -1 && current == 0);
        busy = 0;
        current = 1;
        CHECK(layer(a, nullptr) == FT_OK);
        CHECK(ft_workspace_destroy(a) == FT_OK && freed_on == 1);
        CHECK(ft_workspace_destroy(a) == FT_ERR_ARG);
    } else if (!strcmp(what, "special")) {
        for (long h = 1; h <= 2; ++h)
            for (auto call : {layer, project, expert}) {
                CHECK(call(a, (void*)h) == FT_ERR_ARG && strstr(ftmoe::err, "created stream"));
                CHECK(call(a, nullptr) == FT_OK);
            }
        CHECK(ftmoe::calls == 6);
    }
    printf("ok\n");
    return 0;
}
"""


@pytest.fixture(scope="module")
def harness(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("workspace")
    src, exe = tmp / "workspace.cpp", tmp / "workspace"
    src.write_text(HARNESS)
    subprocess.check_call([COMPILER, "-std=c++17", "-O1", "-w", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", PKG,
                           "-I", "/opt/rocm/include", str(src), "-o", str(exe), "-pthread"])
    return str(exe)


@pytest.mark.parametrize("what", ["device", "destroyed", "capturing", "special"])
def test_workspace(harness, what):
    r = subprocess.run([harness, what], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", (r.returncode, r.stdout)
