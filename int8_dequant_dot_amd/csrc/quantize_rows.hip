// quantize_rows.hip -- symmetric int8 quantisation of rows (tokens).
//
//     a = max |x[r][c]|,  scale[r] = a / 127,  q[r][c] = rint(x[r][c] * (127 / a))
//
// Both quotients are single f32 roundings, the product another, and rint
// rounds halves to even.  |x| <= a, so the product is at most 127 (1 + 2^-23)
// and q stays in [-127, 127].
//
// Memory bounds it: one read of x, one write of q.  A row is read once into
// registers, 16 bytes a lane and load, and quantised from there once its maximum
// is known; rows that do not fit are read a second time.  The maximum is taken
// over the bits of |x|, which order as the values do with infinities and NaN
// above them, so one integer maximum also tells whether the row is finite.
// 8191 x 28672 bfloat16: 110 to 121 us, 6.4 to 5.8 TB/s (the first form, which read
// x twice and stored words one by one: 415 us), float32 186 us; one row of 8192: 2.5 us.
#include "ffn_common.hpp"

namespace loom {

namespace {

// 16 bytes of a row, aligned to its elements.
typedef uint32_t Words __attribute__((ext_vector_type(4)));
typedef Words Words4 __attribute__((aligned(4)));
typedef Words Words2 __attribute__((aligned(2)));
template <int TYPE> struct Chunk {
    static constexpr int kElements = 8;
    typedef Words2 Loose;
};
template <> struct Chunk<LOOM_F32> {
    static constexpr int kElements = 4;
    typedef Words4 Loose;
};

template <int TYPE>
__device__ __forceinline__ float element(const uint32_t (&w)[4], int i) {
    if constexpr (TYPE == LOOM_F32) return __builtin_bit_cast(float, w[i]);
    else if constexpr (TYPE == LOOM_BF16)
        return __builtin_bit_cast(float, i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    else
        return (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i / 2] >> (16 * (i % 2))));
}

// The larger of the magnitudes' bits, by 16-bit halves for 16-bit types.
template <int TYPE>
__device__ __forceinline__ uint32_t larger(uint32_t top, uint32_t w) {
    if constexpr (TYPE == LOOM_F32) return max(top, w & 0x7FFFFFFFu);
    typedef uint16_t Pair __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(Pair, top),
                                                                  __builtin_bit_cast(Pair, w & 0x7FFF7FFFu)));
}

// Chunk c of a row, zeros past its end (a row of a 16-bit type may end with half
// a chunk).
template <int TYPE, bool ONCE>
__device__ __forceinline__ void load_chunk(const typename ElementOf<TYPE>::type *row, int64_t c, int64_t cols,
                                           uint32_t (&w)[4]) {
    constexpr int E = Chunk<TYPE>::kElements;
    const int64_t left = cols - c * E;
    if (left >= E) {
        typedef typename Chunk<TYPE>::Loose Loose;
        const Words v =
            ONCE ? __builtin_nontemporal_load((const Loose *)(row + c * E)) : *(const Loose *)(row + c * E);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = v[i];
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = 0;
        if (E == 8 && left == 4) {
            const uint16_t *half = (const uint16_t *)(row + c * E);
            w[0] = half[0] | (uint32_t)half[1] << 16;
            w[1] = half[2] | (uint32_t)half[3] << 16;
        }
    }
}

// rint(x * inverse) of a chunk: adding 1.5 * 2^23 rounds to a whole number, even
// on ties, and leaves it in the low byte.
template <int TYPE>
__device__ __forceinline__ void store_chunk(int32_t *q, int64_t c, int64_t cols, const uint32_t (&w)[4], float inverse,
                                            bool live) {
    constexpr int E = Chunk<TYPE>::kElements;
    const int64_t left = cols - c * E;
    if (left <= 0) return;
    uint32_t out[E / 4];
#pragma unroll
    for (int j = 0; j < E / 4; ++j) {
        uint32_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            b[i] = __builtin_bit_cast(uint32_t, element<TYPE>(w, 4 * j + i) * inverse + 12582912.0f);
        const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
        out[j] = live ? lo | hi : 0u;
    }
    int32_t *to = q + c * (E / 4);
    if constexpr (E == 4) {
        to[0] = (int32_t)out[0];
    } else if (left >= 8) {
        typedef uint32_t Two __attribute__((ext_vector_type(2), aligned(4)));
        *(Two *)to = Two{out[0], out[1]};
    } else {
        to[0] = (int32_t)out[0];
    }
}

struct RowScale {
    float inverse, scale;
    bool live;
};
template <int TYPE>
__device__ __forceinline__ RowScale scale_of(uint32_t bits) {
    float top;
    if constexpr (TYPE == LOOM_F32) {
        top = __builtin_bit_cast(float, bits);
    } else {
        const uint32_t one = max(bits & 0xFFFFu, bits >> 16);
        const uint32_t w[4] = {one, 0, 0, 0};
        top = element<TYPE>(w, 0);
    }
    const bool finite = top <= 3.4028234663852886e38f, live = finite && top >= kQuantizeTiny;
    return RowScale{live ? 127.0f / top : 0.0f, !finite ? __builtin_nanf("") : live ? top / 127.0f : 0.0f, live};
}

template <int TYPE>
__device__ __forceinline__ uint32_t wave_larger(uint32_t top) {
#pragma unroll
    for (int far = 1; far < kWave; far *= 2) top = larger<TYPE>(top, (uint32_t)__shfl_xor((int)top, far));
    return top;
}

// WAVES waves a row, KEEP chunks a lane held in registers; one wave a row packs 4
// rows into a workgroup.
template <int TYPE, int WAVES, int KEEP>
__global__ __launch_bounds__(kWave * (WAVES > 1 ? WAVES : kQuantizePacked)) void quantize_rows_kernel(
    const typename ElementOf<TYPE>::type *__restrict__ x, int rows, int64_t cols, int64_t row_stride,
    int32_t *__restrict__ q, float *__restrict__ scale) {
    constexpr int kRows = WAVES > 1 ? 1 : kQuantizePacked, kLanes = kWave * WAVES;
    __shared__ uint32_t peaks[WAVES];
    const int lane = WAVES > 1 ? (int)threadIdx.x : lane_id();
    for (int64_t row = (int64_t)blockIdx.x * kRows + (WAVES > 1 ? 0 : threadIdx.x / kWave); row < rows;
         row += (int64_t)gridDim.x * kRows) {
        const auto *src = x + row * row_stride;
        uint32_t kept[KEEP][4], top = 0;
#pragma unroll
        for (int j = 0; j < KEEP; ++j) load_chunk<TYPE, true>(src, lane + j * kLanes, cols, kept[j]);
#pragma unroll
        for (int j = 0; j < KEEP; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = larger<TYPE>(top, kept[j][i]);
        top = wave_larger<TYPE>(top);
        if constexpr (WAVES > 1) {
            if (lane_id() == 0) peaks[threadIdx.x / kWave] = top;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < WAVES; ++i) top = larger<TYPE>(top, peaks[i]);
            __syncthreads();
        }
        const RowScale s = scale_of<TYPE>(top);
        if (lane == 0) scale[row] = s.scale;
        int32_t *to = q + row * (cols / 4);
#pragma unroll
        for (int j = 0; j < KEEP; ++j) store_chunk<TYPE>(to, lane + j * kLanes, cols, kept[j], s.inverse, s.live);
    }
}

// Rows that the registers of a workgroup cannot hold.
template <int TYPE>
__global__ __launch_bounds__(1024) void quantize_long_rows_kernel(const typename ElementOf<TYPE>::type *__restrict__ x,
                                                                  int rows, int64_t cols, int64_t row_stride,
                                                                  int32_t *__restrict__ q, float *__restrict__ scale) {
    constexpr int E = Chunk<TYPE>::kElements;
    __shared__ uint32_t peaks[16];
    const int64_t chunks = (cols + E - 1) / E;
    for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
        const auto *src = x + row * row_stride;
        uint32_t top = 0, w[4];
        for (int64_t c = threadIdx.x; c < chunks; c += 1024) {
            load_chunk<TYPE, false>(src, c, cols, w);
#pragma unroll
            for (int i = 0; i < 4; ++i) top = larger<TYPE>(top, w[i]);
        }
        top = wave_larger<TYPE>(top);
        if (lane_id() == 0) peaks[threadIdx.x / kWave] = top;
        __syncthreads();
        for (int i = 0; i < 16; ++i) top = larger<TYPE>(top, peaks[i]);
        __syncthreads();
        const RowScale s = scale_of<TYPE>(top);
        if (threadIdx.x == 0) scale[row] = s.scale;
        int32_t *to = q + row * (cols / 4);
        for (int64_t c = threadIdx.x; c < chunks; c += 1024) {
            load_chunk<TYPE, true>(src, c, cols, w);
            store_chunk<TYPE>(to, c, cols, w, s.inverse, s.live);
        }
    }
}

template <int TYPE>
void run(const loom_launch_config &cfg, const void *in, int rows, int64_t cols, int64_t row_stride, int32_t *q,
         float *scale, hipStream_t stream) {
    const auto *x = (const typename ElementOf<TYPE>::type *)in;
    const dim3 grid(cfg.workgroups[0]), block(cfg.workgroup_size[0]);
    constexpr int E = Chunk<TYPE>::kElements;
#define LOOM_QUANTIZE(WAVES, KEEP)                                                                                  \
    hipLaunchKernelGGL((quantize_rows_kernel<TYPE, WAVES, KEEP>), grid, block, 0, stream, x, rows, cols, row_stride, \
                       q, scale)
    const int64_t lanes = kWave * quantize_waves(rows, cols), keep = ((cols + E - 1) / E + lanes - 1) / lanes;
    switch (quantize_waves(rows, cols)) {
        case 1:
            if (keep <= 1) LOOM_QUANTIZE(1, 1);
            else if (keep <= 2) LOOM_QUANTIZE(1, 2);
            else LOOM_QUANTIZE(1, 4);
            break;
        case 4:
            if (keep <= 2) LOOM_QUANTIZE(4, 2);
            else if (keep <= 4) LOOM_QUANTIZE(4, 4);
            else LOOM_QUANTIZE(4, 8);
            break;
        case 8:
            if (keep <= 4) LOOM_QUANTIZE(8, 4);
            else LOOM_QUANTIZE(8, 8);
            break;
        default:
            if (keep <= 1) LOOM_QUANTIZE(16, 1);
            else if (keep <= 2) LOOM_QUANTIZE(16, 2);
            else if (keep <= 4) LOOM_QUANTIZE(16, 4);
            else if (cols <= quantize_kept_columns(TYPE)) LOOM_QUANTIZE(16, 8);
            else
                hipLaunchKernelGGL((quantize_long_rows_kernel<TYPE>), grid, block, 0, stream, x, rows, cols, row_stride,
                                   q, scale);
    }
#undef LOOM_QUANTIZE
}

}  // namespace

hipError_t launch_quantize_rows(const loom_launch_config &cfg, const void *x, int type, int rows, int64_t cols,
                                int64_t row_stride, int32_t *q, float *scale, hipStream_t stream) {
    if (type == LOOM_F32) run<LOOM_F32>(cfg, x, rows, cols, row_stride, q, scale, stream);
    else if (type == LOOM_F16) run<LOOM_F16>(cfg, x, rows, cols, row_stride, q, scale, stream);
    else run<LOOM_BF16>(cfg, x, rows, cols, row_stride, q, scale, stream);
    return hipGetLastError();
}

}  // namespace loom
