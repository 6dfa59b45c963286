// Dropout whose mask is computed, never stored, joined to the residual stream.
//
//   y = residual + (keep ? x / (1 - p) : 0)
// keep of element e: half-word e % 8 (low half of a word first) of block e / 8 is
// not below round(65536 p).  A block is the four words of Philox4x32 with ten
// rounds (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", 2011), counter (block, offset), key `seed`.  The gradient is the
// same map without the residual.
//
// HBM bounds it where the generator stays below the memory's time: ten rounds of
// two 64-bit products serve eight elements, a thread's own.  128 x 721 x 1440 bf16
// joined to a residual: 132 us, 6.0 TB/s; a float32 gradient of 16383 x 2047: 53 us,
// 5.1 TB/s.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "disco_internal.h"
#include "vector_io.h"

namespace disco {

namespace {

constexpr int64_t kMostThreads = (int64_t)1 << 31;   // of a launch

struct Words {
    uint32_t w[4];
};

__device__ __forceinline__ Words philox(uint64_t block, uint64_t offset, uint32_t k0, uint32_t k1) {
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
        c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
        c1 = (uint32_t)b;
        c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
        c3 = (uint32_t)a;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return {{c0, c1, c2, c3}};
}

template <typename TX, typename TY, bool RES>
__global__ __launch_bounds__(256) void dropout(const TX* x, const TX* res, TY* y, int64_t n, uint32_t threshold, float scale,
                                               uint64_t seed, uint64_t offset, const int64_t* step, int64_t first) {
    if (step) offset += (uint64_t)*step;
    const int64_t block = first + (int64_t)blockIdx.x * 256 + threadIdx.x, e0 = block * 8;
    if (e0 >= n) return;
    const Words r = philox((uint64_t)block, offset, (uint32_t)seed, (uint32_t)(seed >> 32));
    float f[8], q[8];
    if (e0 + 8 <= n) {
        load_v<TX, 8>(x + e0, f);
        if constexpr (RES) load_v<TX, 8>(res + e0, q);
    } else {
        for (int i = 0; i < 8; ++i) {
            f[i] = e0 + i < n ? load_f(x, e0 + i) : 0.0f;
            if constexpr (RES) q[i] = e0 + i < n ? load_f(res, e0 + i) : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t half = (r.w[i / 2] >> (16 * (i & 1))) & 0xffffu;
        f[i] = half >= threshold ? f[i] * scale : 0.0f;   // whatever x holds there
        if constexpr (RES) f[i] += q[i];
    }
    if (e0 + 8 <= n) {
        store_v<TY, 8>(y + e0, f);
    } else {
        for (int i = 0; i < 8; ++i)
            if (e0 + i < n) store_f(y, e0 + i, f[i]);
    }
}

template <typename TX, typename TY>
int go(const DropoutCall& c, hipStream_t st) {
    const float scale = (float)(65536.0 / (65536 - c.threshold));
    KernelTimer timer("dropout", st);
    for (int64_t first = 0; first * 8 < c.n; first += kMostThreads) {
        const unsigned grid = (unsigned)((std::min(c.n - first * 8, kMostThreads * 8) + 2047) / 2048);
        if (c.residual)
            dropout<TX, TY, true><<<grid, 256, 0, st>>>((const TX*)c.x, (const TX*)c.residual, (TY*)c.y, c.n, c.threshold,
                                                        scale, c.seed, c.offset, c.step, first);
        else
            dropout<TX, TY, false><<<grid, 256, 0, st>>>((const TX*)c.x, nullptr, (TY*)c.y, c.n, c.threshold, scale, c.seed,
                                                         c.offset, c.step, first);
    }
    const hipError_t e = hipGetLastError();
    if (e == hipSuccess) return DISCO_OK;
    return set_error(DISCO_EHIP, "dropout: launch failed: %s", hipGetErrorString(e));
}

}  // namespace

int launch_dropout(const DropoutCall& c, void* stream) {
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (c.x_dtype == DISCO_F32) return c.y_dtype == DISCO_F32 ? go<float, float>(c, st) : go<float, bf16_t>(c, st);
    return c.y_dtype == DISCO_F32 ? go<bf16_t, float>(c, st) : go<bf16_t, bf16_t>(c, st);
}

}  // namespace disco
