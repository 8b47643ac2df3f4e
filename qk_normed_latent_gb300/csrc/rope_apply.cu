// qkmla_rope: rotary positions on RoPE blocks that lie in memory on their own or inside a head.
//
// Pair i of a block, at position p, turns by p f_i:  (a, b) -> (a cos - b sin, a sin + b cos),
// its two elements neighbours (interleaved) or d_r / 2 apart (halves).  f_i is theta^(-2i/d_r), for a
// longer context divided by a factor -- all pairs (linear), or the slow ones and not the fast ones
// (YaRN: pairs of more than beta_fast turns within the original context keep their frequency, of less
// than beta_slow are divided, a ramp between) -- or given.
//
// Angles.  The host forms each frequency in turns a position, in 64 bits (to 2^-48 of itself: neighbours by products, up to seven
// behind a power), and hands the kernel its fraction as a 64-bit integer F (unit 2^-64 turns): p F modulo 2^64 is the angle modulo one turn, by one
// integer product, for every int32 position.  Read as a signed number it is the turn nearest 0, so that a
// small angle keeps its relative precision; sincospif takes it from there.
//
// Bound: HBM, each element read and written once (3 flops an element).  A block of 256 threads takes whole
// rows, up to four vectors (or pairs of them) a thread: their loads go out first, and while they are on their way
// the block forms the rows' cosines and sines once in shared memory, for every head.  Vectors stay as they lie in
// memory until they are turned: as fp32 from the start they took twice the registers, and 4096 x 128 RoPE blocks of
// 64 bf16 values 38.4 us where this takes 23.4 (134 MB: 5.7 TB/s).  16 x 16 blocks of 32 take 3 us, a launch and one
// chain of loads, 16001 fp32 keys of 64 4.6 (4.3 while the next launch could start early).  16-byte accesses where strides, bases and d_r allow them, else one pair at a time.
#include <cmath>
#include <cstdlib>

#include "common.cuh"

namespace qkmla {
namespace {

constexpr int kMaxPairs = 128;
constexpr int kThreadsR = 256;
constexpr int kItems = 4;                  // vectors (or pairs of them) a thread has in flight
constexpr int kTable = 2048;               // cosines a block keeps

struct RopeParams {
    uint64_t turn[kMaxPairs];              // frequency of a pair, in 2^-64 turns
    const void* x;
    void* out;
    const int32_t* positions;
    int64_t xr, xh, yr, yh;                // strides in elements
    int rows, heads, pairs, rows_per_block, heads_per_block;
    float gain, sign;
};

// V elements as they lie in memory: 16 bytes, or V of them one by one.
template <typename T> constexpr int kFull = 16 / (int)sizeof(T);
template <typename T, int V> struct Held {
    alignas(V == kFull<T> ? 16 : alignof(T)) T e[V];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (V == kFull<T>) *reinterpret_cast<uint4*>(e) = *reinterpret_cast<const uint4*>(p);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) e[i] = p[i];
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (V == kFull<T>) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(e);
        else
#pragma unroll
            for (int i = 0; i < V; ++i) p[i] = e[i];
    }
};

// One unit of work: V neighbouring elements (interleaved: V / 2 pairs), or V elements of each half
// (V pairs).  V = 2 and 1 for the two layouts where 16-byte accesses are not possible.
template <typename T, bool HALF, int V>
__global__ void __launch_bounds__(kThreadsR) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int kPairs = HALF ? V : V / 2;
    __shared__ float cs[kTable], sn[kTable];
    __shared__ uint64_t freq[kMaxPairs];
    const int r0 = blockIdx.x * p.rows_per_block;
    const int nr = min(p.rows_per_block, p.rows - r0);
    const int h0 = blockIdx.y * p.heads_per_block;
    const int nh = min(p.heads_per_block, p.heads - h0);
    const int units = p.pairs / kPairs;                 // a head's
    const int n = nr * nh * units;                      // at most kThreadsR * kItems
    // A warp's 32 frequencies are 32 addresses in constant memory, which serves one at a time.  Where a thread has more
    // than one angle they are copied out of it once (16001 keys of 64, calls in a row that overlapped: 7.0 us without, 4.2 with; 4096 x 128 blocks, two rows
    // a block: 23.35 and 23.6).
    const bool many = nr * p.pairs > kThreadsR;
    if (many) {
        for (int i = threadIdx.x; i < p.pairs; i += kThreadsR) freq[i] = p.turn[i];
        __syncthreads();
    }
    pdl_wait();                                         // (no early launch of the next kernel: append reads new tokens ahead of its wait)
    Held<T, V> a[kItems], b[HALF ? kItems : 1];
    int at[kItems];
    int64_t to[kItems];
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        const int k = threadIdx.x + j * kThreadsR;
        at[j] = -1;
        if (k >= n) continue;
        const int u = k % units, rh = k / units;
        const int r = rh / nh, h = rh - r * nh;
        const T* x = (const T*)p.x + (int64_t)(r0 + r) * p.xr + (int64_t)(h0 + h) * p.xh + u * V;
        at[j] = r * p.pairs + u * kPairs;
        to[j] = (int64_t)(r0 + r) * p.yr + (int64_t)(h0 + h) * p.yh + u * V;
        a[j].load(x);
        if constexpr (HALF) b[j].load(x + p.pairs);
    }
    for (int k = threadIdx.x; k < nr * p.pairs; k += kThreadsR) {
        const int r = k / p.pairs, i = k - r * p.pairs;
        const int64_t turn = (int64_t)((uint64_t)(int64_t)p.positions[r0 + r] * (many ? freq[i] : p.turn[i]));
        float s, c;
        sincospif((float)turn * 1.0842021724855044e-19f, &s, &c);   // 2^-63: sin and cos of pi x take half turns
        cs[k] = c * p.gain;
        sn[k] = s * p.gain * p.sign;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kItems; ++j) {
        if (at[j] < 0) continue;
#pragma unroll
        for (int i = 0; i < kPairs; ++i) {
            const float c = cs[at[j] + i], s = sn[at[j] + i];
            T *u, *v;
            if constexpr (HALF) { u = &a[j].e[i]; v = &b[j].e[i]; }
            else { u = &a[j].e[2 * i]; v = &a[j].e[2 * i + 1]; }
            const float x = Elem<T>::load(u), y = Elem<T>::load(v);
            Elem<T>::store(u, fmaf(-y, s, x * c));
            Elem<T>::store(v, fmaf(x, s, y * c));
        }
        T* y = (T*)p.out + to[j];
        a[j].store(y);
        if constexpr (HALF) b[j].store(y + p.pairs);
    }
}

// Frequencies in radians a position, in 64 bits; false for arguments that have none.
bool frequencies(const qkmla_rope_args* a, double* f) {
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    const int n = a->d_r / 2;
    if (a->scaling == QKMLA_ROPE_GIVEN) {
        for (int i = 0; i < n; ++i) {
            f[i] = a->frequencies[i];
            if (!std::isfinite(f[i])) return false;
        }
        return true;
    }
    const double step = std::pow((double)a->theta, -2.0 / a->d_r);
    f[0] = 1.0;
    for (int i = 1; i < n; ++i) f[i] = i % 8 ? f[i - 1] * step : std::pow((double)a->theta, -2.0 * i / a->d_r);
    if (a->scaling == QKMLA_ROPE_LINEAR)
        for (int i = 0; i < n; ++i) f[i] /= (double)a->factor;
    if (a->scaling == QKMLA_ROPE_YARN) {
        // the (fractional) pair that makes `turns` turns within the original context
        const double l = 2.0 * std::log((double)a->theta);
        auto pair_of = [&](double turns) { return a->d_r * std::log(a->original_context / (turns * kTwoPi)) / l; };
        const double low = std::fmax(std::floor(pair_of(a->beta_fast)), 0.0);
        const double high = std::fmin(std::ceil(pair_of(a->beta_slow)), a->d_r - 1.0);
        const double width = std::fmax(high - low, 0.001);
        for (int i = 0; i < n; ++i) {
            const double ramp = std::fmin(std::fmax((i - low) / width, 0.0), 1.0);
            f[i] = f[i] / (double)a->factor * ramp + f[i] * (1.0 - ramp);
        }
    }
    return true;
}

template <typename T, bool HALF, int V>
int launch_rope(RopeParams& p, cudaStream_t s) {
    // whole rows a block while a thread has fewer than kItems units; many heads of one row are cut
    const int units = p.pairs / (HALF ? V : V / 2);
    const int want = kThreadsR * kItems;
    p.heads_per_block = min(p.heads, max(1, want / units));
    p.rows_per_block = max(1, min(min(want / (units * p.heads_per_block), kTable / p.pairs), p.rows));
    // few rows: one a block, so that a step's call uses more SMs (its cosines then cost more than its copies)
    while (p.rows_per_block > 1 && (p.rows + p.rows_per_block - 1) / p.rows_per_block < 2 * device_sm_count())
        p.rows_per_block = (p.rows_per_block + 1) / 2;
    const int64_t gx = ((int64_t)p.rows + p.rows_per_block - 1) / p.rows_per_block;
    const int gy = (p.heads + p.heads_per_block - 1) / p.heads_per_block;
    if (gy > 65535) return QKMLA_ERR_UNSUPPORTED;
    return launch_pdl(rope_kernel<T, HALF, V>, dim3((unsigned)gx, gy), dim3(kThreadsR), 0, s, p) == cudaSuccess
               ? QKMLA_OK
               : QKMLA_ERR_CUDA;
}

template <typename T>
int launch_rope_type(RopeParams& p, bool half, bool vec, cudaStream_t s) {
    constexpr int F = kFull<T>;
    if (half) return vec ? launch_rope<T, true, F>(p, s) : launch_rope<T, true, 1>(p, s);
    return vec ? launch_rope<T, false, F>(p, s) : launch_rope<T, false, 2>(p, s);
}

}  // namespace
}  // namespace qkmla

using namespace qkmla;

extern "C" int qkmla_rope(const qkmla_rope_args* a, void* stream) {
    if (!a || a->rows < 0 || a->heads < 1 || a->d_r < 2 || a->d_r % 2) return QKMLA_ERR_INVALID;
    if (a->layout != QKMLA_ROPE_INTERLEAVED && a->layout != QKMLA_ROPE_HALVES) return QKMLA_ERR_INVALID;
    if (a->scaling < QKMLA_ROPE_PLAIN || a->scaling > QKMLA_ROPE_GIVEN) return QKMLA_ERR_INVALID;
    if (a->scaling == QKMLA_ROPE_GIVEN) {
        if (!a->frequencies) return QKMLA_ERR_INVALID;
    } else if (!(a->theta > 1.f) || !std::isfinite(a->theta)) {
        return QKMLA_ERR_INVALID;
    }
    if (a->scaling == QKMLA_ROPE_LINEAR || a->scaling == QKMLA_ROPE_YARN)
        if (!(a->factor > 0.f) || !std::isfinite(a->factor)) return QKMLA_ERR_INVALID;
    if (a->scaling == QKMLA_ROPE_YARN)
        if (a->original_context < 1 || !(a->beta_slow > 0.f) || !(a->beta_fast >= a->beta_slow) || !std::isfinite(a->beta_fast))
            return QKMLA_ERR_INVALID;
    if (!std::isfinite(a->attention_factor) || a->attention_factor < 0.f) return QKMLA_ERR_INVALID;
    if (a->dtype != QKMLA_F32 && a->dtype != QKMLA_BF16) return QKMLA_ERR_UNSUPPORTED;
    if (a->d_r > 2 * kMaxPairs) return QKMLA_ERR_UNSUPPORTED;
    if (a->rows == 0) return QKMLA_OK;
    // rows or heads that share elements of the output would be written (in place: read and written) by several threads
    if ((a->rows > 1 && std::llabs(a->out_row_stride) < a->d_r) || (a->heads > 1 && std::llabs(a->out_head_stride) < a->d_r))
        return QKMLA_ERR_INVALID;
    if (!a->x || !a->out || !a->positions) return QKMLA_ERR_INVALID;
    const int esz = a->dtype == QKMLA_F32 ? 4 : 2;
    if ((uintptr_t)a->x % esz || (uintptr_t)a->out % esz || (uintptr_t)a->positions % 4) return QKMLA_ERR_INVALID;
    RopeParams p;
    double f[kMaxPairs];
    if (!frequencies(a, f)) return QKMLA_ERR_INVALID;
    p.pairs = a->d_r / 2;
    for (int i = 0; i < p.pairs; ++i) {
        double turn = std::fabs(f[i]) * 0.15915494309189533576888376337251;       // 1 / (2 pi)
        turn -= std::floor(turn);                                      // exact, in [0, 1)
        const uint64_t n = (uint64_t)(turn * 18446744073709551616.0);
        p.turn[i] = f[i] < 0.0 ? 0 - n : n;                            // (1 - turn would drop bits of a small one)
    }
    p.x = a->x;
    p.out = a->out;
    p.positions = a->positions;
    p.xr = a->x_row_stride;
    p.xh = a->x_head_stride;
    p.yr = a->out_row_stride;
    p.yh = a->out_head_stride;
    p.rows = a->rows;
    p.heads = a->heads;
    p.gain = a->attention_factor == 0.f ? 1.f : a->attention_factor;
    p.sign = a->inverse ? -1.f : 1.f;
    const bool half = a->layout == QKMLA_ROPE_HALVES;
    const int F = 16 / esz;
    bool vec = (half ? p.pairs % F : a->d_r % F) == 0 && (uintptr_t)a->x % 16 == 0 && (uintptr_t)a->out % 16 == 0;
    for (int64_t st : {p.xr, p.xh, p.yr, p.yh}) vec = vec && st % F == 0;
    cudaStream_t s = (cudaStream_t)stream;
    return a->dtype == QKMLA_F32 ? launch_rope_type<float>(p, half, vec, s)
                                 : launch_rope_type<__nv_bfloat16>(p, half, vec, s);
}
