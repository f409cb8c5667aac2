// What the appends that rotate by position share (rope.cu, norm_rope.cu): rows as
// raw words, E4M3 codes of a few values, the cosine and sine of an angle.
#pragma once

#include "device_utils.cuh"

namespace pkv {

namespace {

constexpr int kThreads = 128;  // kMaxRopePairs: a thread makes one cosine and sine at most

// V elements of T as raw words.
template <int kBytes>
struct Raw {
    static constexpr int kWords = kBytes >= 4 ? kBytes / 4 : 1;
    uint32_t w[kWords];
    __device__ __forceinline__ void load(const char* p) {
        if constexpr (kBytes == 16) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
        } else if constexpr (kBytes == 8) {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            w[0] = v.x, w[1] = v.y;
        } else if constexpr (kBytes == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else if constexpr (kBytes == 2) {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint8_t*>(p);
        }
    }
    __device__ __forceinline__ void store(char* p) const {
        if constexpr (kBytes == 16)
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        else if constexpr (kBytes == 8)
            *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
        else if constexpr (kBytes == 4)
            *reinterpret_cast<uint32_t*>(p) = w[0];
        else if constexpr (kBytes == 2)
            *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(w[0]);
        else
            *reinterpret_cast<uint8_t*>(p) = static_cast<uint8_t>(w[0]);
    }
};

template <int DT, int V>
__device__ __forceinline__ void unpack(const Raw<V * static_cast<int>(sizeof(typename Elem<DT>::T))>& r, float* f) {
    using T = typename Elem<DT>::T;
    const T* e = reinterpret_cast<const T*>(r.w);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = Elem<DT>::to_float(e[i]);
}

template <int DT, int V>
__device__ __forceinline__ Raw<V * static_cast<int>(sizeof(typename Elem<DT>::T))> pack(const float* f) {
    using T = typename Elem<DT>::T;
    Raw<V * static_cast<int>(sizeof(T))> r;
    T* e = reinterpret_cast<T*>(r.w);
#pragma unroll
    for (int i = 0; i < V; ++i) e[i] = Elem<DT>::from_float(f[i]);
    return r;
}

// E4M3 codes of V values / scale (as kv_append_fp8).
template <int V>
__device__ __forceinline__ Raw<V> quantize(const float* f, float scale) {
    Raw<V> r;
    if constexpr (V == 1) {
        r.w[0] = e4m3x2_from_floats(__fdiv_rn(f[0], scale), 0.f) & 0xFFu;
    } else {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            const uint32_t c = e4m3x2_from_floats(__fdiv_rn(f[2 * i], scale), __fdiv_rn(f[2 * i + 1], scale));
            if (i & 1)
                r.w[i / 2] |= c << 16;
            else
                r.w[i / 2] = c;
        }
    }
    return r;
}

// Cosine and sine of `turn` (a fraction of a turn times 2^64, as a signed
// number), times `amplitude`.
__device__ __forceinline__ float2 rotor(uint64_t turn, float amplitude) {
    const int32_t t = static_cast<int32_t>((turn + 0x80000000ull) >> 32);  // to 2^-32 of a turn, nearest
    const uint32_t quarter = (static_cast<uint32_t>(t) + 0x20000000u) >> 30;
    const int32_t rest = static_cast<int32_t>(static_cast<uint32_t>(t) - (quarter << 30));  // at most 2^29
    float s, c;
    sincospif(static_cast<float>(rest) * 0x1p-31f, &s, &c);
    const float cq = (quarter & 1u) ? s : c, sq = (quarter & 1u) ? c : s;
    // Quarter turns 1 and 2 flip the cosine's sign, 2 and 3 the sine's.
    const float cs = (quarter == 1u || quarter == 2u) ? -cq : cq;
    const float sn = quarter >= 2u ? -sq : sq;
    return make_float2(cs * amplitude, sn * amplitude);
}

}  // namespace

}  // namespace pkv
