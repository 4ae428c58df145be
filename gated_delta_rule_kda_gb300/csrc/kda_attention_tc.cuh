// What the tensor-core attention kernels share: tiles of 128 rows and 128 keys, the ring of k, v
// stages, the products of one row tile, the split of a CTA's 384 threads.
#pragma once

#include "kda_common.cuh"
#include "tc_primitives.cuh"

namespace kda {
namespace attn_tc {

using namespace tc;

constexpr int kThreads = 384;
constexpr int kTile = 128;                    // rows of a row tile, keys of a key tile
constexpr uint32_t kTileBytes = kTile * kD * 2;
constexpr int kStages = 5;
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpScrub = 11;
// 384 threads start with 168 registers; the softmax warps take 208, the others keep 88:
// 256 * 208 + 128 * 88 = 384 * 168
constexpr int kRegsSoftmax = 208, kRegsOther = 88;

// (a.x + b.x, a.y + b.y)
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    return fma2(a, make_float2(1.f, 1.f), b);
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const void *tmap, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// The ring of k, v stages: tile loads in order, stage n % kStages, phase n / kStages.  A load
// completes B_KVFULL of its stage, or B_RAW when the tile is values to be gone through first
// (B_CLEAN follows); those barriers' phases are counted by use, a bit a stage.
struct Ring {
    int stage = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next() {
        if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
        }
    }
};

// One 128-wide product is eight MMAs of 64 cycles each, all issued by one thread: their matrix
// descriptors differ from the first one's by constants (16-byte units of the address field).
__device__ __forceinline__ void mma_scores(uint32_t tmem, uint64_t q_desc, uint64_t k_desc, int r, int from, int to) {
#pragma unroll
    for (int s = from; s < to; ++s) {
        const uint64_t step = ((s >> 2) * (kTileBytes / 2) + (s & 3) * 32) / 16;
        mma_bf16(tmem + 128 * r, q_desc + step, k_desc + step, idesc_bf16_f32(kTile, kTile), s > 0);
    }
}
// Keys 64 half .. 64 half + 63 of a tile.
__device__ __forceinline__ void mma_values(uint32_t tmem, uint64_t v_desc, int r, int half, bool first) {
#pragma unroll
    for (int s = 4 * half; s < 4 * half + 4; ++s)
        mma_bf16_tmem_a(tmem + 256 + 128 * r, tmem + 128 * r + 8 * s, v_desc + s * (2048 / 16),
                        idesc_bf16_f32(kTile, kD) | kIdescBMN, s > 0 ? 1u : !first);
}

constexpr uint32_t kMinusInf = 0xff800000u;

__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
    float a = __uint_as_float(s[0]), b = __uint_as_float(s[1]);
#pragma unroll
    for (int k = 2; k < 30; k += 4) {
        a = fmaxf(fmaxf(a, __uint_as_float(s[k])), __uint_as_float(s[k + 1]));
        b = fmaxf(fmaxf(b, __uint_as_float(s[k + 2])), __uint_as_float(s[k + 3]));
    }
    return fmaxf(fmaxf(a, b), fmaxf(__uint_as_float(s[30]), __uint_as_float(s[31])));
}

}  // namespace attn_tc
}  // namespace kda
