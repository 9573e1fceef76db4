"""Which decode calls need the driver's tensor-map encoder: those whose kernels copy by tensor maps.  The
4-bit cache's kernel copies runs of memory, so its calls go through without one.

The library's argument and dispatch code (gqa_decode.o of the build) is linked with stand-ins for the CUDA
calls it makes and for the kernels' launches; nothing is launched or dereferenced.
"""
import ctypes
import os
import subprocess

import pytest

import decode_attention_gb300 as gqa
from decode_attention_gb300 import build

FAKES = r"""
#include <cstddef>
namespace gqa {
struct LaunchArgs;
int launches = 0;
int launch_sliding(const LaunchArgs&, bool) { ++launches; return 0; }
int launch_global(const LaunchArgs&, bool) { ++launches; return 0; }
int launch_global_keqv(const LaunchArgs&, bool) { ++launches; return 0; }
int launch_keqv_tc(const LaunchArgs&, bool) { ++launches; return 0; }
int launch_mq(const LaunchArgs&, bool, bool) { ++launches; return 0; }
int launch_quant(const LaunchArgs&, bool, bool) { ++launches; return 0; }
int launch_nibble(const LaunchArgs&, bool, bool) { ++launches; return 0; }
int mq_max_queries(bool) { return 4; }
}
static int encoder;
static void *registered;
extern "C" {
void set_encoder(int on) { encoder = on; }
int launch_count() { return gqa::launches; }
int cudaGetDevice(int *dev) { *dev = 0; return 0; }
int cudaDeviceGetAttribute(int *value, int, int) { *value = 152; return 0; }
int cudaGetDriverEntryPointByVersion(const char *, void **fn, unsigned, unsigned long long, int *found) {
    *fn = encoder ? reinterpret_cast<void *>(&launch_count) : nullptr;   // (never called)
    *found = encoder ? 0 : 1;
    return 0;
}
int cudaMalloc(void **, size_t) { return 2; }
int cudaFree(void *) { return 0; }
int cudaMemcpy(void *, const void *, size_t, int) { return 2; }
int cudaMemsetAsync(void *, int, size_t, void *) { return 0; }
int cudaStreamSynchronize(void *) { return 0; }
void **__cudaRegisterFatBinary(void *) { return &registered; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
}
"""
F = 0x10000   # aligned address, never dereferenced
SLIDING, GLOBAL = (32, 16, 256), (32, 4, 512)


def linked(tmp_path):
    gqa.load_library()
    obj = os.path.join(build.BUILD_DIR, "gqa_decode.o")
    if not os.path.exists(obj):
        build.build(force=True)
    (tmp_path / "fakes.cpp").write_text(FAKES)
    so = str(tmp_path / "dispatch.so")
    subprocess.run(["g++", "-shared", "-fPIC", "-O1", "-Wl,-Bsymbolic", str(tmp_path / "fakes.cpp"), obj, "-o", so,
                    "-lpthread"], check=True)
    lib = ctypes.CDLL(so, mode=os.RTLD_LOCAL | os.RTLD_NOW)
    real, vp = gqa.load_library(), ctypes.c_void_p
    for name in ("gqa_decode", "gqa_decode_nibble", "gqa_decode_nibble_paged", "gqa_decode_quant"):
        getattr(lib, name).argtypes = getattr(real, name).argtypes
    assert real.gqa_decode.argtypes[0] is vp
    return lib


@pytest.mark.parametrize("encoder", [0, 1])
@pytest.mark.parametrize("H,KVH,D", [SLIDING, GLOBAL])
def test_who_needs_tensor_maps(tmp_path, encoder, H, KVH, D):
    lib = linked(tmp_path)
    lib.set_encoder(encoder)
    ws = (F, 1 << 30)
    mapped = gqa.GQA_OK if encoder else gqa.GQA_ERR_CUDA
    assert lib.gqa_decode(F, F, F, F, 2, 64, H, KVH, D, 0, F, 0, *ws, None) == mapped
    assert lib.gqa_decode_quant(F, F, F, F, F, F, 2, 64, H, KVH, D, 0, F, 0, *ws, None) == mapped
    assert lib.launch_count() == 2 * encoder
    assert lib.gqa_decode_nibble(F, F, F, 2, 64, H, KVH, D, 0, F, 0, *ws, None) == gqa.GQA_OK
    assert lib.gqa_decode_nibble_paged(F, F, F, F, 2, 8, 4, 16, H, KVH, D, 0, F, 0, *ws, None) == gqa.GQA_OK
    assert lib.launch_count() == 2 * encoder + 2
    assert lib.gqa_decode_nibble(F, F, F, 2, 64, H, KVH, D, 0, F, 0, F, 16, None) == gqa.GQA_ERR_WORKSPACE
