// sv_sort.h -- bitonic ordering of one value per lane, without LDS inside a
// wave, and the k-th largest value of a workgroup.
#pragma once

#include "sv_device.h"

namespace sv {

// Compare-exchange partners: lane ^ MASK by DPP for masks within 16 lanes
// (half-row and row mirrors are ^ 7 and ^ 15, a rotation by 8 is ^ 8, and the
// half-row mirror after the quad's is ^ 4); across rows and halves the swap
// of a register with itself gives both rows' values to every lane.
template <int MASK>
__device__ __forceinline__ int lane_xor(int v)
{
    static_assert(MASK == 1 || MASK == 2 || MASK == 3 || MASK == 4 || MASK == 7 || MASK == 8 || MASK == 15 ||
                      MASK == 16 || MASK == 31 || MASK == 32 || MASK == 63,
                  "partner of a bitonic step");
    const int lane = threadIdx.x & 63;
    if (MASK == 1) return dpp_int<kDppQuadXor1>(v);
    if (MASK == 2) return dpp_int<kDppQuadXor2>(v);
    if (MASK == 3) return dpp_int<0x1B>(v);
    if (MASK == 4) return dpp_int<kDppRowHalfMirror>(dpp_int<0x1B>(v));
    if (MASK == 7) return dpp_int<kDppRowHalfMirror>(v);
    if (MASK == 8) return dpp_int<0x128>(v);
    if (MASK == 15) return dpp_int<kDppRowMirror>(v);
    if (MASK == 31 || MASK == 63) v = dpp_int<kDppRowMirror>(v);
    if (MASK != 32) {
        const IntPair p = swap_halves<16>(v);
        v = (lane & 16) ? p.a : p.b;
    }
    if (MASK == 32 || MASK == 63) {
        const IntPair p = swap_halves<32>(v);
        v = (lane & 32) ? p.a : p.b;
    }
    return v;
}

template <int MASK>
__device__ __forceinline__ float lane_xor(float v)
{
    return __int_as_float(lane_xor<MASK>(__float_as_int(v)));
}

template <int MASK>
__device__ __forceinline__ double lane_xor(double v)
{
    return __hiloint2double(lane_xor<MASK>(__double2hiint(v)), lane_xor<MASK>(__double2loint(v)));
}

template <int MASK>
__device__ __forceinline__ uint64_t lane_xor(uint64_t v)
{
    const uint32_t lo = (uint32_t)lane_xor<MASK>((int)(uint32_t)v);
    const uint32_t hi = (uint32_t)lane_xor<MASK>((int)(uint32_t)(v >> 32));
    return ((uint64_t)hi << 32) | lo;
}

__device__ __forceinline__ float larger(float x, float y) { return fmaxf(x, y); }
__device__ __forceinline__ float smaller(float x, float y) { return fminf(x, y); }
__device__ __forceinline__ uint64_t larger(uint64_t x, uint64_t y) { return x > y ? x : y; }
__device__ __forceinline__ uint64_t smaller(uint64_t x, uint64_t y) { return x > y ? y : x; }

// One step: of each pair (lane, lane ^ MASK) the lane without bit BIT keeps
// the larger value.
template <int MASK, int BIT, class T>
__device__ __forceinline__ T sort_step(T v)
{
    const T w = lane_xor<MASK>(v);
    const T hi = larger(v, w), lo = smaller(v, w);
    return ((int)threadIdx.x & BIT) ? lo : hi;
}

// A bitonic sequence over the 64 lanes into descending order.
template <class T>
__device__ __forceinline__ T wave_merge(T v)
{
    v = sort_step<32, 32>(v);
    v = sort_step<16, 16>(v);
    v = sort_step<8, 8>(v);
    v = sort_step<4, 4>(v);
    v = sort_step<2, 2>(v);
    return sort_step<1, 1>(v);
}

// The wave's 64 values in descending lane order.
template <class T>
__device__ __forceinline__ T wave_sort(T v)
{
    v = sort_step<1, 1>(v);
    v = sort_step<3, 2>(v);
    v = sort_step<1, 1>(v);
    v = sort_step<7, 4>(v);
    v = sort_step<2, 2>(v);
    v = sort_step<1, 1>(v);
    v = sort_step<15, 8>(v);
    v = sort_step<4, 4>(v);
    v = sort_step<2, 2>(v);
    v = sort_step<1, 1>(v);
    v = sort_step<31, 16>(v);
    v = sort_step<8, 8>(v);
    v = sort_step<4, 4>(v);
    v = sort_step<2, 2>(v);
    v = sort_step<1, 1>(v);
    v = sort_step<63, 32>(v);
    v = sort_step<16, 16>(v);
    v = sort_step<8, 8>(v);
    v = sort_step<4, 4>(v);
    v = sort_step<2, 2>(v);
    return sort_step<1, 1>(v);
}

// The k-th largest (1 <= k <= 64) of the values of the workgroup's first
// kBlock threads, one each; every thread calls it and gets the result.
// Every wave sorts its 64; the larger of a descending list and a reversed one
// are the best 64 of both and bitonic, so two merges leave the best 64 of
// all.  lds: kBlock + 1 values, free again after the call.
template <class T>
__device__ __forceinline__ T block_kth(T v, int k, T *lds)
{
    static_assert(kWaves == 4, "two levels of merges");
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    if (wave < kWaves) lds[threadIdx.x] = v = wave_sort(v);
    __syncthreads();
    if (wave < 2) {
        v = wave_merge(larger(lds[wave * 128 + lane], lds[wave * 128 + 127 - lane]));
        if (wave == 1) lds[128 + lane] = v;
    }
    __syncthreads();
    if (wave == 0) {
        v = wave_merge(larger(v, lds[128 + 63 - lane]));
        if (lane == k - 1) lds[kBlock] = v;
    }
    __syncthreads();
    v = lds[kBlock];
    __syncthreads();
    return v;
}

}  // namespace sv
