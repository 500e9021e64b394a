// Norm of queries and keys for each head, their position rotation, and the store of keys and values
// into the paged cache: one pass, each value read once and written once.
//
// 16 lanes hold one head of one token, lane c the dims c NE .. c NE + NE - 1 (NE = head_dim / 16), so
// a head row is one contiguous 16-lane access and the mean of squares is a 16-lane butterfly. Pairs
// (2 i, 2 i + 1) lie in one lane; pairs (i, i + rot / 2) are rot / 2 / NE lanes apart (rot a multiple
// of head_dim / 8, so that the distance is whole) and come by lane shuffles. The cosines and sines of
// a token are computed once per workgroup into LDS: the angle is position * inv_freq in fp64, reduced
// to a fraction of a turn there (at position 10^6 an fp32 angle would be off by 0.03), and only the
// fraction goes to fp32.
// Bound: HBM for prompts (319 MB read and written in 69 us, 4.6 TB/s; a plain copy of this card reaches
// 4.9), launch and memory latency for a few tokens (3.3 us for one).
#include "cache_internal.h"

namespace ubw {
namespace cache {
namespace {

using h16 = _Float16;
using b16 = __bf16;

template <typename T, int N>
struct alignas(N * sizeof(T) < 16 ? N * sizeof(T) : 16) Vec {
    T x[N];
};

template <typename T, int NE>
__device__ inline void load_row(const T* p, float (&x)[NE]) {
    const Vec<T, NE> v = *reinterpret_cast<const Vec<T, NE>*>(p);
#pragma unroll
    for (int i = 0; i < NE; ++i) x[i] = (float)v.x[i];
}
template <typename T, int NE>
__device__ inline void store_row(T* p, const float (&x)[NE]) {
    Vec<T, NE> v;
#pragma unroll
    for (int i = 0; i < NE; ++i) v.x[i] = (T)x[i];
    *reinterpret_cast<Vec<T, NE>*>(p) = v;
}
// NE values to e4m3, rounded to nearest even by the conversion instruction. It turns what is too
// large into NaN, so values are cut at the largest one first; a NaN passes.
template <int NE>
__device__ inline void store_e4m3(char* p, const float (&x)[NE], float scale) {
    Vec<uint32_t, NE / 4> v;
#pragma unroll
    for (int i = 0; i < NE; i += 4) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float z = x[i + j] / scale;
            y[j] = z != z ? z : fminf(fmaxf(z, -448.f), 448.f);
        }
        int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
        v.x[i / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
    }
    *reinterpret_cast<Vec<uint32_t, NE / 4>*>(p) = v;
}
// The output types are launch constants: a uniform branch at the store instead of more instances.
template <int NE>
__device__ inline void store_as(int dtype, char* row, int first, const float (&x)[NE], const float* scale) {
    if (dtype == UBW_F16)
        store_row<h16, NE>(reinterpret_cast<h16*>(row) + first, x);
    else if (dtype == UBW_BF16)
        store_row<b16, NE>(reinterpret_cast<b16*>(row) + first, x);
    else
        store_e4m3<NE>(row + first, x, scale ? *scale : 1.f);
}

// cos and sin of turn i of the token's rotation
__device__ inline float2 turn(int position, float freq) {
    const double r = (double)position * (double)freq * 0.15915494309189533576888;  // turns
    const float f = (float)(r - rint(r));
    float2 cs;
    sincospif(2.f * f, &cs.y, &cs.x);
    return cs;
}

template <typename TI, int D, bool PAIRS>
__global__ __launch_bounds__(256) void k_rope(RopeArgs a, int heads_per_wg) {
    constexpr int NE = D / 16;
    __shared__ float2 cs[D / 2];
    const int t = blockIdx.x;
    const int half = a.rot >> 1;
    const int position = a.positions[t];
    const int slot = a.slots[t];
    if ((int)threadIdx.x < half) cs[threadIdx.x] = turn(position, a.inv_freq[threadIdx.x]);
    __syncthreads();

    const int lane = threadIdx.x & 15;
    const int kvh = a.c.heads;
    const int all = a.heads + 2 * kvh;
    const int h0 = blockIdx.y * heads_per_wg;
    const int h1 = min(all, h0 + heads_per_wg);
    const bool stored = (uint32_t)slot < ((uint32_t)a.c.pages << a.c.lps);
    const int64_t page = slot >> a.c.lps;
    const uint32_t row = (uint32_t)slot & ((1u << a.c.lps) - 1);

    // rotated pairs of this lane: cosine and signed sine per element (identity past rot)
    const int d0 = lane * NE;
    float co[NE], si[NE];
    int partner = threadIdx.x & 63;
    if constexpr (PAIRS) {
#pragma unroll
        for (int i = 0; i < NE; i += 2) {
            const bool in = d0 + i < a.rot;
            const float2 c = in ? cs[(d0 + i) >> 1] : make_float2(1.f, 0.f);
            co[i] = co[i + 1] = c.x;
            si[i] = -c.y;
            si[i + 1] = c.y;
        }
    } else {
        const bool low = d0 < half, in = d0 < a.rot;
        partner += in ? (low ? half / NE : -(half / NE)) : 0;
#pragma unroll
        for (int i = 0; i < NE; ++i) {
            const float2 c = in ? cs[low ? d0 + i : d0 + i - half] : make_float2(1.f, 0.f);
            co[i] = c.x;
            si[i] = low ? -c.y : c.y;
        }
    }

    for (int hb = h0; hb < h1; hb += 16) {
        const int h = hb + (threadIdx.x >> 4);
        const bool live = h < h1;
        const bool isq = h < a.heads, isv = h >= a.heads + kvh;
        const int hh = isq ? h : isv ? h - a.heads - kvh : h - a.heads;
        const TI* src = static_cast<const TI*>(isq ? a.q : isv ? a.v : a.k) + t * (isq ? a.ldq : isv ? a.ldv : a.ldk) +
                        (int64_t)hh * D + d0;
        float x[NE];
        if (live) {
            load_row<TI, NE>(src, x);
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] = 0.f;
        }
        const float* w = isv ? nullptr : isq ? a.qw : a.kw;
        if (w && live) {
            const auto mean_square = [&] {
                float ss = 0.f;
#pragma unroll
                for (int i = 0; i < NE; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
                for (int m = 1; m < 16; m <<= 1) ss += __shfl_xor(ss, m, 16);
                return ss * (1.f / D);
            };
            float mean = mean_square() + a.eps;
            if (!(mean > 1e-30f && mean < 1e38f)) {
                // squares near the ends of fp32 (alike in a head's 16 lanes): of x 2^-e, with eps 2^-2e, where the
                // larger of them comes near 1
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < NE; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
                for (int m = 1; m < 16; m <<= 1) top = fmaxf(top, __shfl_xor(top, m, 16));
                int e = __builtin_amdgcn_frexp_expf(top);
                if (a.eps > 0.f) e = max(e, (__builtin_amdgcn_frexp_expf(a.eps) + 1) >> 1);
#pragma unroll
                for (int i = 0; i < NE; ++i) x[i] = ldexpf(x[i], -e);
                mean = mean_square() + ldexpf(a.eps, -2 * e);
            }
            const float r = 1.f / sqrtf(mean);
            float g[NE];
            load_row<float, NE>(w + d0, g);
#pragma unroll
            for (int i = 0; i < NE; ++i) x[i] = x[i] * r * g[i];
        }
        // every lane takes part in the exchange, values and padding heads keep what they hold
        float z[NE];
        if constexpr (PAIRS) {
#pragma unroll
            for (int i = 0; i < NE; i += 2) {
                z[i] = fmaf(x[i], co[i], x[i + 1] * si[i]);
                z[i + 1] = fmaf(x[i + 1], co[i + 1], x[i] * si[i + 1]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NE; ++i) z[i] = fmaf(x[i], co[i], __shfl(x[i], partner) * si[i]);
        }
        const bool turned = !isv && d0 < a.rot;
        if (!turned) {
#pragma unroll
            for (int i = 0; i < NE; ++i) z[i] = x[i];
        } else if (PAIRS && d0 + NE > a.rot) {  // rot ends inside the lane
#pragma unroll
            for (int i = 0; i < NE; ++i)
                if (d0 + i >= a.rot) z[i] = x[i];
        }
        if (!live) continue;
        if (isq) {
            store_as<NE>(a.out_dtype, static_cast<char*>(a.out) + (t * a.ldo + (int64_t)h * D) * 2, d0, z, nullptr);
        } else if (stored) {
            char* at = isv ? a.c.v + page * a.c.v_page + hh * a.c.v_head + (int64_t)row * a.c.v_row
                           : a.c.k + page * a.c.k_page + hh * a.c.k_head + (int64_t)row * a.c.k_row;
            const float* sc = isv ? a.c.v_scale : a.c.k_scale;
            store_as<NE>(a.cache_dtype, at, d0, z, sc ? sc + hh : nullptr);
        }
    }
}

template <typename TI, int D>
hipError_t launch(const RopeArgs& a, bool pairs, hipStream_t s) {
    const int all = a.heads + 2 * a.c.heads;
    // One pass of 16 heads per workgroup while there are few, else all heads of a token, its angles
    // computed once (8191 tokens of 80 heads: 69 us, 77 with 32 heads a workgroup, 87 with 16).
    const int per = (int64_t)a.tokens * cdiv(all, 16) <= 2048 ? 16 : (int)cdiv(all, 16) * 16;
    const dim3 grid(a.tokens, (unsigned)cdiv(all, per));
    if (pairs)
        k_rope<TI, D, true><<<grid, 256, 0, s>>>(a, per);
    else
        k_rope<TI, D, false><<<grid, 256, 0, s>>>(a, per);
    return hipGetLastError();
}
template <typename TI>
hipError_t launch_d(const RopeArgs& a, int d, bool pairs, hipStream_t s) {
    return d == 64 ? launch<TI, 64>(a, pairs, s) : d == 128 ? launch<TI, 128>(a, pairs, s) : launch<TI, 256>(a, pairs, s);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& a, int in_dtype, int head_dim, bool interleaved, hipStream_t s) {
    return in_dtype == UBW_F32   ? launch_d<float>(a, head_dim, interleaved, s)
           : in_dtype == UBW_F16 ? launch_d<h16>(a, head_dim, interleaved, s)
                                 : launch_d<b16>(a, head_dim, interleaved, s);
}

}  // namespace cache
}  // namespace ubw
