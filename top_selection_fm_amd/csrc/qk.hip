// qk.hip -- norms of queries and keys for each head, the position rotation in the same pass, and
// the keys and values written into the pages of a cache.
//
// For a head's values x (D of them) at position p:
//   y = x / sqrt(mean(x^2) + eps) * g,   pairs (a, b) of the rotated dims -> (a c - b s, a s + b c),
// c, s of the angle p theta_i (YaRN's theta, formed on the host in float64).  Everything between
// the load and the store is float32, so q, k and v are rounded once, at the store: to bf16, or for
// 132-byte rows to e4m3 codes of x / scale with scale = max |x| / 448.
//
// Bound by memory (each value is read and written once), for single tokens by launch latency.  A
// workgroup takes one row: D / VEC lanes hold a head, VEC values (16 bytes) each, so a wave has 2
// to 8 heads at once and the norm is a few lane swaps.  The row's angles are formed once, one
// pair a thread, and shared through LDS by all its heads: p theta / 2 pi is reduced to a fraction
// of a turn in float64 (positions reach millions), the sine and cosine of that are float32.
// 4,096 rows of 32 + 8 + 8 heads of 128 into fp8 pages: 26 us, 3.6 TB/s of the 4.84 that a large
// copy reaches; 32 rows of 64 + 8 + 8 heads: 4.5 us, 7.7 with the launch.
#include "fm_internal.h"

namespace fm {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

template <bool F32> struct Io {
    static constexpr int VEC = F32 ? 4 : 8, SIZE = F32 ? 4 : 2;
    __device__ static __forceinline__ u32x4 raw(const void *p, int64_t at) {
        return *(const u32x4 *)((const uint8_t *)p + at * SIZE);
    }
    __device__ static __forceinline__ void widen(float *x, const u32x4 &r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F32) {
                x[i] = __uint_as_float(r[i]);
            } else {
                x[2 * i] = __uint_as_float(r[i] << 16);
                x[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
            }
        }
    }
    __device__ static __forceinline__ void store(const float *x, void *p, int64_t at) {
        u32x4 r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (F32) {
                r[i] = __float_as_uint(x[i]);
            } else {
                const f32x2 v = {x[2 * i], x[2 * i + 1]};
                r[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
            }
        }
        *(u32x4 *)((uint8_t *)p + at * SIZE) = r;
    }
};

template <int L> __device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) x += __shfl_xor(x, o);
    return x;
}
template <int L> __device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
    for (int o = 1; o < L; o <<= 1) x = fmaxf(x, __shfl_xor(x, o));
    return x;
}

template <bool F32, int D>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(QkArgs A) {
    using IO = Io<F32>;
    constexpr int VEC = IO::VEC, L = D / VEC, GROUPS = 256 / L;
    __shared__ float2 cs[FM_HEAD_DIM / 2];
    const int t = blockIdx.x, tid = threadIdx.x, lane = tid % L, e0 = VEC * lane;
    const int half = A.rope_dim / 2;
    const int heads = A.n_heads + A.n_kv * (A.store ? 2 : 1), by = gridDim.y * GROUPS;
    // head i of the row: q's, then k's, then v's
    auto fetch = [&](int i) {
        const bool is_q = i < A.n_heads, is_v = i >= A.n_heads + A.n_kv;
        const int h = is_q ? i : is_v ? i - A.n_heads - A.n_kv : i - A.n_heads;
        return IO::raw(is_q ? A.q : is_v ? A.v : A.k, t * (is_q ? A.q_ld : is_v ? A.v_ld : A.k_ld) + (int64_t)h * D + e0);
    };
    // the first head and the weights are on their way while the angles are formed
    int i = blockIdx.y * GROUPS + tid / L;
    u32x4 next = {0u, 0u, 0u, 0u}, qw = next, kw = next;
    if (i < heads) next = fetch(i);
    if (A.q_norm) qw = IO::raw(A.q_norm, e0);
    if (A.k_norm) kw = IO::raw(A.k_norm, e0);
    if (tid < half) {
        double turns = (double)A.pos[t] * A.turns[tid];
        turns -= rint(turns);
        float s, c;
        sincospif(2.f * (float)turns, &s, &c);
        cs[tid] = make_float2(c, s);
    }
    // where the row's entry goes
    int64_t cell = -1;
    if (A.store) {
        const int b = A.row_req ? A.row_req[t] : A.b_is_zero ? 0 : t;
        if (b >= 0 && b < A.B) {
            const int slot = A.slot ? A.slot[t] : A.pos[t];
            if (slot >= 0 && slot < min(A.seq_lens[b], A.max_len)) {
                const int page = A.bt[(int64_t)b * A.bt_ld + slot / kPage];
                if (page >= 0 && page < A.n_phys) cell = (int64_t)page * A.n_kv * kPage + slot % kPage;
            }
        }
    }
    __syncthreads();
    const bool turned = e0 >= A.rope_first && e0 < A.rope_first + A.rope_dim;
    for (; i < heads; i += by) {
        float x[VEC];
        IO::widen(x, next);
        if (i + by < heads) next = fetch(i + by);
        const bool is_q = i < A.n_heads, is_v = i >= A.n_heads + A.n_kv;
        const int h = is_q ? i : is_v ? i - A.n_heads - A.n_kv : i - A.n_heads;
        if (is_v && cell < 0) continue;
        if (!is_v) {
            if (is_q ? A.q_norm : A.k_norm) {
                float w[VEC], ss = 0.f;
                IO::widen(w, is_q ? qw : kw);
#pragma unroll
                for (int j = 0; j < VEC; ++j) ss = fmaf(x[j], x[j], ss);
                const float inv = 1.0f / sqrtf(lanes_sum<L>(ss) / (float)D + A.eps);
#pragma unroll
                for (int j = 0; j < VEC; ++j) x[j] *= inv * w[j];
            }
            if (A.halves) {
                // the pair's other value sits half / VEC lanes away (the dims are multiples of VEC)
                const int r = e0 - A.rope_first;
                const bool upper = r >= half;
                const int from = turned ? (upper ? lane - half / VEC : lane + half / VEC) : lane;
                float y[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[j] = __shfl(x[j], from, L);
                if (turned) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const float2 a = cs[(upper ? r - half : r) + j];
                        x[j] = upper ? y[j] * a.y + x[j] * a.x : x[j] * a.x - y[j] * a.y;
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < VEC; j += 2) {
                    const int r = e0 + j - A.rope_first;
                    if (r >= 0 && r < A.rope_dim) {
                        const float2 a = cs[r / 2];
                        const float u = x[j], v = x[j + 1];
                        x[j] = u * a.x - v * a.y;
                        x[j + 1] = u * a.y + v * a.x;
                    }
                }
            }
            if (is_q) {
                IO::store(x, A.q_out, t * A.q_out_ld + (int64_t)h * D + e0);
                continue;
            }
            if (A.k_out) IO::store(x, A.k_out, t * A.k_out_ld + (int64_t)h * D + e0);
        }
        if (cell < 0) continue;
        uint8_t *pool = (uint8_t *)(is_v ? A.v_pool : A.k_pool);
        const int64_t row = cell + (int64_t)h * kPage;
        if (F32 || !A.fp8) {
            IO::store(x, pool, row * D + e0);
        } else if constexpr (!F32 && D == kDim) {
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < VEC; ++j) top = fmaxf(top, fabsf(x[j]));
            top = lanes_max<L>(top);
            const float scale = top > 0.f ? top / 448.f : 1.f;
            u32x2 codes;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float y[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) y[k] = fminf(fmaxf(x[4 * j + k] / scale, -448.f), 448.f);
                int w = __builtin_amdgcn_cvt_pk_fp8_f32(y[0], y[1], 0, false);
                codes[j] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y[2], y[3], w, true);
            }
            uint32_t *to = (uint32_t *)(pool + row * kRowFp8);     // rows are 4-byte aligned
            to[2 * lane] = codes[0];
            to[2 * lane + 1] = codes[1];
            if (lane == 0) to[kDim / 4] = __float_as_uint(scale);
        }
    }
}

}  // namespace

hipError_t launch_qk(const QkArgs &a, bool f32, int head_dim, hipStream_t s) {
    // few rows: a row's heads go to several workgroups, as many as leave every group of lanes one;
    // many rows fill the chip by themselves, and a row's angles are then formed once
    const int lanes = head_dim / (f32 ? 4 : 8), groups = 256 / lanes;
    const int heads = a.n_heads + a.n_kv * (a.store ? 2 : 1);
    const int parts = a.T >= 1024 ? 1 : (heads + groups - 1) / groups;
    const dim3 grid((unsigned)a.T, (unsigned)parts);
    if (f32 && head_dim == 64) qk_norm_rope_kernel<true, 64><<<grid, 256, 0, s>>>(a);
    else if (f32) qk_norm_rope_kernel<true, 128><<<grid, 256, 0, s>>>(a);
    else if (head_dim == 64) qk_norm_rope_kernel<false, 64><<<grid, 256, 0, s>>>(a);
    else qk_norm_rope_kernel<false, 128><<<grid, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace fm
