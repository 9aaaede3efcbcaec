// layer_norm_bwd.cu -- layer norm backward (include/swiglu_ops.h).
//
// Bound by HBM: a row is read once into shared memory, a row ahead, and its gradient written
// once; the arithmetic of its columns runs in packed pairs, as forward, and the column sums stay
// in registers until the last row.  Measured, 11136 x 3584 bf16 with the residual stream's
// gradient, 319 MB: 57 us, 5.6 TB/s of the 6.78 TB/s of a copy.
#include "layer_norm.cuh"

namespace swiglu {
namespace {

constexpr int kBwdThreads = 384;

struct NormBwd {
    const void *dy, *s, *gamma, *skip;
    const float *mean, *rstd;
    void* dx;
    float *pg, *pb;                // partial planes [gridDim][D] of dgamma and dbeta (NULL: not wanted)
    int64_t lddy, lds, ldk, lddx, M;
    int D, lanes, gf32;
};

// ---------------------------------------------------------------- rows on their way

// 16 bytes, of which `bytes` are read and the rest are zero.
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, int bytes = 16) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void commit_async() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_async() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row read and the next one in flight, in shared memory, filled by asynchronous copies.  A
// thread copies and reads its own packs, so this needs no barrier.  Layout:
// [tensor][stage][pack][thread].
constexpr int kStages = 2;

template <class T, int NV>
struct Rows {
    const char* next = nullptr;            // this lane's pack 0 of the row to copy
    int64_t hop = 0;                       // bytes from a group's row to its next
    uint32_t slot = 0;                     // shared address of this thread's slot, stage 0, pack 0
    uint32_t per = 0;                      // bytes from a pack's slots to the next pack's
    __device__ __forceinline__ void init(const T* base, int64_t ld, int64_t row, int64_t step, int lane, uint32_t smem,
                                         int tensor) {
        next = reinterpret_cast<const char*>(base + row * ld) + lane * 16;
        hop = step * ld * (int64_t)sizeof(T);
        per = blockDim.x * 16;
        slot = smem + tensor * kStages * NV * per + threadIdx.x * 16;
    }
    // Copies the group's next row into a stage; `lane16`: 16 x lane, `pitch`: 16 x lanes.
    __device__ __forceinline__ void issue(int stage, int lane16, int pitch, int row_bytes) {
        const uint32_t to = slot + stage * NV * per;
#pragma unroll
        for (int q = 0; q < NV; ++q)
            if (q < NV - 1 || q * pitch + lane16 < row_bytes) copy_async(to + q * per, next + q * pitch);
        next += hop;
    }
    // The same for the first and the last row of a tensor, [lo, hi), which shifted packs overhang.
    __device__ __forceinline__ void issue_within(int stage, int lane16, int pitch, int row_bytes, uintptr_t lo, uintptr_t hi) {
        const uint32_t to = slot + stage * NV * per;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const uintptr_t from = reinterpret_cast<uintptr_t>(next + q * pitch);
            if (q == NV - 1 && q * pitch + lane16 >= row_bytes) continue;
            if (from >= lo) {
                copy_async(to + q * per, next + q * pitch, from + 16 <= hi ? 16 : (int)(hi - from));
            } else {
                store_smem(to + q * per, load_edge<T>(reinterpret_cast<const T*>(lo), -(int)((lo - from) / sizeof(T)), kVec<T>));
            }
        }
        next += hop;
    }
    // Pack q of a stage, once its copies have landed.
    __device__ __forceinline__ uint4 get(int stage, int q) const { return load_smem(slot + (stage * NV + q) * per); }
    // Zeros in place of its elements that are not the row's.
    __device__ __forceinline__ void trim(int stage, int q, int first, int D) const {
        store_smem(slot + (stage * NV + q) * per, row_elements<T>(get(stage, q), first, D));
    }
};

// Two sums at once.  The first exchange leaves the low half-warp with x and the high half
// with y, so that the two take 5 or 6 shuffles instead of 10.
__device__ __forceinline__ float2 row_sum2(float2 v, int group, int lanes, float2* red, int buf) {
    const bool high = threadIdx.x & 16;
    float t = (high ? v.y : v.x) + __shfl_xor_sync(0xffffffffu, high ? v.x : v.y, 16);
#pragma unroll
    for (int o = 8; o; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    if (lanes == 32) {
        const float u = __shfl_xor_sync(0xffffffffu, t, 16);
        return high ? make_float2(u, t) : make_float2(t, u);
    }
    red += buf * kRed;
    if ((threadIdx.x & 15) == 0) reinterpret_cast<float*>(&red[(threadIdx.x - group * lanes) >> 5])[high] = t;
    group_sync(group, lanes);
    v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kRed; w += 2) {
        if (w * 32 >= lanes) break;
        const float4 f = *reinterpret_cast<const float4*>(red + w);
        v.x += f.x + f.z;
        v.y += f.y + f.w;
    }
    return v;
}

// ---------------------------------------------------------------- backward

// The row's two sums, dx, and fp32 column sums of dy * xh and dy over the group's rows, kept
// in registers; the CTA's groups are added in shared memory at the end and written once, as
// this CTA's partial planes.  A row is read from the ring twice, before and after the
// reduction, which costs less than keeping xh and g beside the column sums.  (With one row
// ahead in registers instead of the ring it took 92 us of 11136 x 3584 bf16.)
// xh = (s - mean) * rstd, whose difference loses nothing however far the mean is from 0 (a product
// -mean * rstd rounded on its own would put |mean| * rstd * 2^-24 into every xh of the row), and
// dx = g * rstd + xh * A + B with A = -c2 * rstd, B = -c1 * rstd.
// Shared memory: red [groups][2][kRed] pairs, gamma (whole packs, fp32), then the rows in
// flight, and after them the groups' column sums in their place.
template <class T, int NV, bool SKIP, bool EDGE>
__global__ void __launch_bounds__(kBwdThreads) layer_norm_bwd_kernel(const NormBwd a) {
    constexpr int V = kVec<T>, P = V / 2;
    extern __shared__ uint4 smem[];
    const int lanes = a.lanes, lane = threadIdx.x % lanes, group = threadIdx.x / lanes, D = a.D;
    const int rows = blockDim.x / lanes, width = padded(EDGE ? D + V - 1 : D);
    float2* red = reinterpret_cast<float2*>(smem) + group * 2 * kRed;
    float* gamma = reinterpret_cast<float*>(smem) + rows * 4 * kRed + (EDGE ? group * width : 0);
    float* acc = reinterpret_cast<float*>(smem) + rows * 4 * kRed + (EDGE ? rows : 1) * width;
    const int64_t step = (int64_t)gridDim.x * rows;
    int64_t row = (int64_t)blockIdx.x * rows + group;
    // a group's rows lie alike: it has one, or they are a multiple of 152 rows, of whole packs, apart
    const int m = EDGE ? into_pack<T>(a.s, row, a.lds) : 0, end = D + m;
    const int lane16 = lane * 16, pitch = lanes * 16, row_bytes = end * (int)sizeof(T);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(acc);
    Rows<T, NV> dy, s, skip;
    dy.init(static_cast<const T*>(a.dy) - m, a.lddy, row, step, lane, ring, 0);
    s.init(static_cast<const T*>(a.s) - m, a.lds, row, step, lane, ring, 1);
    if (SKIP) skip.init(static_cast<const T*>(a.skip) - m, a.ldk, row, step, lane, ring, 2);
    auto issue = [&](int stage, int64_t i) {
        if (EDGE && (i == 0 || i == a.M - 1)) {
            auto within = [&](Rows<T, NV>& t, const void* base, int64_t ld) {
                const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
                t.issue_within(stage, lane16, pitch, row_bytes, lo, lo + (uintptr_t)((a.M - 1) * ld + D) * sizeof(T));
            };
            within(dy, a.dy, a.lddy);
            within(s, a.s, a.lds);
            if (SKIP) within(skip, a.skip, a.ldk);
        } else if (i < a.M) {
            dy.issue(stage, lane16, pitch, row_bytes);
            s.issue(stage, lane16, pitch, row_bytes);
            if (SKIP) skip.issue(stage, lane16, pitch, row_bytes);
        }
        commit_async();
    };
    cudaTriggerProgrammaticLaunchCompletion();             // the parameters' kernel may come up meanwhile
    issue(0, row);
    for (int i = threadIdx.x; i < rows * 4 * kRed; i += blockDim.x) reinterpret_cast<float*>(smem)[i] = 0.f;
    if (EDGE) stage_param<T>(gamma, a.gamma, a.gf32, D, m, width, 1.f, lane, lanes);
    else stage_param<T>(gamma, a.gamma, a.gf32, D, 0, width, 1.f, threadIdx.x, blockDim.x);
    const uint32_t gamma_at = (uint32_t)__cvta_generic_to_shared(gamma);
    __syncthreads();
    F2 dg[NV * P], db[NV * P];
#pragma unroll
    for (int i = 0; i < NV * P; ++i) dg[i] = db[i] = f2(0.f);
    float mean = 0.f, rstd = 0.f;
    if (row < a.M) mean = a.mean[row], rstd = a.rstd[row];
    const float inv = 1.f / (float)D;
    for (int stage = 0; row < a.M; row += step, stage ^= 1) {
        issue(stage ^ 1, row + step);
        const float mu = mean, rs = rstd;
        if (row + step < a.M) mean = a.mean[row + step], rstd = a.rstd[row + step];
        wait_async<1>();
        if (EDGE) {
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                const int k = q * lanes + lane;
                if (on_edge<T, NV>(q, k, m, end) && in_row<T, NV>(q, k, end)) {
                    dy.trim(stage, q, k * V - m, D);
                    s.trim(stage, q, k * V - m, D);
                }
            }
        }
        const F2 rs2 = f2(rs), centre = f2(-mu);
        F2 c1 = f2(0.f), c2 = f2(0.f);
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int k = q * lanes + lane;
            if (in_row<T, NV>(q, k, end)) {
                F2 w[P], d[P], xs[P];
                load_staged<T>(w, gamma_at, k, width);
                unpack16<T>(dy.get(stage, q), d);
                unpack16<T>(s.get(stage, q), xs);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const F2 xh = (xs[i] + centre) * rs2, g = d[i] * w[i];
                    dg[q * P + i] = fma(d[i], xh, dg[q * P + i]);
                    db[q * P + i] = db[q * P + i] + d[i];
                    c1 = c1 + g;
                    c2 = fma(g, xh, c2);
                }
            }
        }
        const float2 p1 = split(c1), p2 = split(c2);
        float2 c = row_sum2(make_float2(p1.x + p1.y, p2.x + p2.y), group, lanes, red, stage);
        c.x *= inv * rs;
        c.y *= inv * rs;
        const F2 A = f2(-c.y), B = f2(-c.x);
        T* o = static_cast<T*>(a.dx) + row * a.lddx - m;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int k = q * lanes + lane;
            if (in_row<T, NV>(q, k, end)) {
                F2 w[P], d[P], xs[P];
                load_staged<T>(w, gamma_at, k, width);
                unpack16<T>(dy.get(stage, q), d);
                unpack16<T>(s.get(stage, q), xs);
#pragma unroll
                for (int i = 0; i < P; ++i) w[i] = fma(d[i] * w[i], rs2, fma((xs[i] + centre) * rs2, A, B));
                if (SKIP) {
                    unpack16<T>(skip.get(stage, q), d);
#pragma unroll
                    for (int i = 0; i < P; ++i) w[i] = w[i] + d[i];
                }
                if (EDGE && on_edge<T, NV>(q, k, m, end)) store_edge<T>(o + m, k * V - m, D, pack16<T>(w));
                else reinterpret_cast<uint4*>(o)[k] = pack16<T>(w);
            }
        }
    }
    if (a.pg == nullptr && a.pb == nullptr) return;
    // the groups' sums meet in the ring's place: [group][2][columns, 16-byte pieces of packs apart]
    wait_async<0>();
    __syncthreads();
    const int half = sizeof(T) == 2 ? width / 2 : 0;
    float* mine = acc + group * 2 * width;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        const int k = q * lanes + lane;
        if (in_row<T, NV>(q, k, end)) {
#pragma unroll
            for (int h = 0; h < P / 2; ++h) {
                const float2 g0 = split(dg[q * P + 2 * h]), g1 = split(dg[q * P + 2 * h + 1]);
                const float2 b0 = split(db[q * P + 2 * h]), b1 = split(db[q * P + 2 * h + 1]);
                reinterpret_cast<float4*>(mine + h * half)[k] = make_float4(g0.x, g0.y, g1.x, g1.y);
                reinterpret_cast<float4*>(mine + width + h * half)[k] = make_float4(b0.x, b0.y, b1.x, b1.y);
            }
        }
    }
    __syncthreads();
    auto place = [&](int c) { return sizeof(T) == 4 ? c : (c & 4 ? half : 0) + (c >> 3) * 4 + (c & 3); };
    const int first = EDGE ? into_pack<T>(a.s, (int64_t)blockIdx.x * rows, a.lds) : 0;
    constexpr int kAtOnce = 4;             // columns a thread adds at a time
    for (int c0 = threadIdx.x; c0 < D; c0 += kAtOnce * blockDim.x) {
        float g[kAtOnce], b[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) g[j] = b[j] = 0.f;
        for (int w = 0; w < rows; ++w) {
            const float* p = acc + w * 2 * width;
            const int at = EDGE ? (first + w * (int)(a.lds & (V - 1))) & (V - 1) : 0;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const int c = c0 + j * blockDim.x;
                if (c < D) g[j] += p[place(c + at)], b[j] += p[width + place(c + at)];
            }
        }
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            const int c = c0 + j * blockDim.x;
            if (c >= D) continue;
            if (a.pg) a.pg[(int64_t)blockIdx.x * D + c] = g[j];
            if (a.pb) a.pb[(int64_t)blockIdx.x * D + c] = b[j];
        }
    }
}

// Rows off 16-byte boundaries, element by element: THREADS threads walk the rows of a worker (a warp, or the CTA),
// whose column sums are its own partial plane.  A row comes to shared memory in the aligned
// 16-byte pieces that cover it, one row ahead, and is read there element by element (loaded
// to registers instead, 2 bytes at a time, it took 207 us where this takes 85 for
// 4864 x 5003 bf16).  It is bound by instructions, 64 a column.  Shared memory: [worker][stage][tensor][pitch bytes].
__host__ __device__ constexpr int narrow_pitch(int row_bytes) { return (row_bytes + 14) / 16 * 16 + 16; }

template <class T>
__device__ __forceinline__ void copy_row(char* to, const T* base, int64_t ld, int64_t i, int64_t M, int D, int t, int threads) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(base), hi = lo + (uintptr_t)((M - 1) * ld + D) * sizeof(T);
    const uintptr_t start = lo + (uintptr_t)(i * ld) * sizeof(T), first = start & ~uintptr_t(15);
    const int pieces = (int)((start + (uintptr_t)D * sizeof(T) - first + 15) / 16);
    for (int p = t; p < pieces; p += threads) {
        const uintptr_t from = first + (uintptr_t)p * 16;
        char* dst = to + p * 16;
        if (from >= lo) {
            copy_async((uint32_t)__cvta_generic_to_shared(dst), reinterpret_cast<const void*>(from),
                       from + 16 <= hi ? 16 : (int)(hi - from));
        } else {                           // the tensor starts inside this piece
            for (uintptr_t e = lo; e < from + 16 && e < hi; e += sizeof(T))
                *reinterpret_cast<T*>(dst + (e - from)) = *reinterpret_cast<const T*>(e);
        }
    }
}

template <class T, bool SKIP, int THREADS>
__global__ void __launch_bounds__(THREADS < 128 ? 128 : THREADS, THREADS > 128 ? 1 : 4)
    layer_norm_bwd_narrow_kernel(const NormBwd a) {
    constexpr int TENSORS = SKIP ? 3 : 2;
    __shared__ __align__(16) float2 red[2 * kRed];
    extern __shared__ uint4 smem[];
    const int t = threadIdx.x % THREADS, D = a.D, pitch = narrow_pitch(D * (int)sizeof(T));
    const int64_t worker = (int64_t)blockIdx.x * (blockDim.x / THREADS) + threadIdx.x / THREADS;
    const int64_t step = (int64_t)gridDim.x * (blockDim.x / THREADS);
    char* rows = reinterpret_cast<char*>(smem) + threadIdx.x / THREADS * 2 * TENSORS * pitch;
    cudaTriggerProgrammaticLaunchCompletion();
    if (THREADS > 32) {
        if (threadIdx.x < 2 * kRed) red[threadIdx.x] = make_float2(0.f, 0.f);
    }
    const T* src[3] = {static_cast<const T*>(a.dy), static_cast<const T*>(a.s), static_cast<const T*>(a.skip)};
    const int64_t ld[3] = {a.lddy, a.lds, a.ldk};
    auto issue = [&](int stage, int64_t i) {
        if (i < a.M) {
#pragma unroll
            for (int k = 0; k < TENSORS; ++k)
                copy_row<T>(rows + (stage * TENSORS + k) * pitch, src[k], ld[k], i, a.M, D, t, THREADS);
        }
        commit_async();
    };
    // this thread's first element of a tensor's row in a stage
    auto at = [&](int stage, int k, int64_t i) {
        const int m = (int)(reinterpret_cast<uintptr_t>(src[k] + i * ld[k]) & 15);
        return reinterpret_cast<const T*>(rows + (stage * TENSORS + k) * pitch + m) + t;
    };
    float dg[kCols], db[kCols];
#pragma unroll
    for (int j = 0; j < kCols; ++j) dg[j] = db[j] = 0.f;
    int64_t row = worker;
    issue(0, row);
    const float inv = 1.f / (float)D;
    for (int stage = 0; row < a.M; row += step, stage ^= 1) {
        const float mu = a.mean[row], rs = a.rstd[row];
        wait_async<0>();
        if (THREADS > 32) group_sync(0, THREADS);          // all pieces are here, and the other stage has been read
        else __syncwarp();
        issue(stage ^ 1, row + step);
        const T *y = at(stage, 0, row), *s = at(stage, 1, row);
        float g[kCols], xh[kCols];
        float2 c = make_float2(0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            if (t + j * THREADS < D) {
                const float d = to_f32(y[j * THREADS]);
                xh[j] = (to_f32(s[j * THREADS]) - mu) * rs;
                g[j] = d * param(a.gamma, a.gf32, t + j * THREADS, 1.f, (T*)nullptr);
                dg[j] += d * xh[j];
                db[j] += d;
                c.x += g[j];
                c.y += g[j] * xh[j];
            }
        }
        c = row_sum2(c, 0, THREADS, red, stage);
        c.x *= inv;
        c.y *= inv;
        T* o = static_cast<T*>(a.dx) + row * a.lddx + t;
        const T* k = at(stage, SKIP ? 2 : 0, row);
#pragma unroll
        for (int j = 0; j < kCols; ++j) {
            if (t + j * THREADS < D) {
                float v = rs * (g[j] - c.x - xh[j] * c.y);
                if (SKIP) v += to_f32(k[j * THREADS]);
                o[j * THREADS] = from_f32<T>(v);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < kCols; ++j) {
        if (t + j * THREADS < D) {
            if (a.pg) a.pg[worker * D + t + j * THREADS] = dg[j];
            if (a.pb) a.pb[worker * D + t + j * THREADS] = db[j];
        }
    }
}

// Rows wider than the registers hold, in two passes: the two sums of every row, then dx
// and the column sums of a block of columns over a range of rows.  Bound by HBM, which reads dy and
// s twice: 3000 x 16384 bf16 with the residual stream's gradient 137 us, 590 MB at 4.3 TB/s; single
// elements, for rows off 16-byte boundaries, 3000 x 14001: 240 us.
template <class T, int VEC>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_bwd_wide_sums_kernel(const NormBwd a, float2* sums) {
    __shared__ __align__(16) float2 red[2 * kRed];
    if (threadIdx.x < 2 * kRed) red[threadIdx.x] = make_float2(0.f, 0.f);
    __syncthreads();
    int buf = 0;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x, buf ^= 1) {
        const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
        const T* s = static_cast<const T*>(a.s) + row * a.lds;
        const float mean = a.mean[row], rstd = a.rstd[row];
        LongSum sum_g, sum_gx;
        constexpr int run = VEC > 1 ? 1 : kRun;
        const int64_t hop = blockDim.x * VEC;
        for (int64_t col = threadIdx.x * VEC; col < a.D;) {
            float2 part = make_float2(0.f, 0.f);
#pragma unroll 1
            for (int i = 0; i < run && col < a.D; ++i, col += hop) {
                float w[VEC], d[VEC], xs[VEC];
                load_pack<T, VEC>(dy + col).unpack(d);
                load_pack<T, VEC>(s + col).unpack(xs);
                load_param<T, VEC>(w, a.gamma, a.gf32, (int)col, 1.f);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float g = d[j] * w[j];
                    part.x += g;
                    part.y += g * ((xs[j] - mean) * rstd);
                }
            }
            sum_g.add(part.x);
            sum_gx.add(part.y);
        }
        const float2 c = row_sum2(make_float2(sum_g.value(), sum_gx.value()), 0, blockDim.x, red, buf);
        if (threadIdx.x == 0) sums[row] = make_float2(c.x / (float)a.D, c.y / (float)a.D);
    }
}

// grid (column blocks, row ranges): CTA (x, y) has columns x * blockDim * VEC ... and rows
// y, y + gridDim.y, ...; its column sums are partial plane y.
template <class T, int VEC>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_bwd_wide_kernel(const NormBwd a, const float2* sums) {
    cudaTriggerProgrammaticLaunchCompletion();
    const int64_t col = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * VEC;
    if (col >= a.D) return;
    float w[VEC], dg[VEC], db[VEC];
    load_param<T, VEC>(w, a.gamma, a.gf32, (int)col, 1.f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) dg[j] = db[j] = 0.f;
    for (int64_t row = blockIdx.y; row < a.M; row += gridDim.y) {
        float d[VEC], xs[VEC];
        load_pack<T, VEC>(static_cast<const T*>(a.dy) + row * a.lddy + col).unpack(d);
        load_pack<T, VEC>(static_cast<const T*>(a.s) + row * a.lds + col).unpack(xs);
        const float mean = a.mean[row], rstd = a.rstd[row];
        const float2 c = sums[row];
        float o[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const float xh = (xs[j] - mean) * rstd;
            dg[j] += d[j] * xh;
            db[j] += d[j];
            o[j] = rstd * (d[j] * w[j] - c.x - xh * c.y);
        }
        if (a.skip) {
            load_pack<T, VEC>(static_cast<const T*>(a.skip) + row * a.ldk + col).unpack(d);
#pragma unroll
            for (int j = 0; j < VEC; ++j) o[j] += d[j];
        }
        store_pack<T, VEC>(static_cast<T*>(a.dx) + row * a.lddx + col, o);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        if (a.pg) a.pg[(int64_t)blockIdx.y * a.D + col + j] = dg[j];
        if (a.pb) a.pb[(int64_t)blockIdx.y * a.D + col + j] = db[j];
    }
}

// dgamma and dbeta: the planes added in plane order (16 strided runs, then the runs).  Its 2 D
// columns of 152 planes are in L2; what it costs is a launch and two rounds of latency, about 4 us.
template <class W>
__global__ void __launch_bounds__(512) layer_norm_params_kernel(const float* pg, const float* pb, W* dgamma, W* dbeta,
                                                                int planes, int D) {
    __shared__ float part[16][33];
    const float* p = blockIdx.y == 0 ? pg : pb;
    W* out = blockIdx.y == 0 ? dgamma : dbeta;
    if (out == nullptr) return;
    const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
    float t = 0.f;
    cudaGridDependencySynchronize();       // launched beside the kernel that writes the planes
    if (col < D) {
#pragma unroll 10
        for (int i = threadIdx.y; i < planes; i += 16) t += p[(int64_t)i * D + col];
    }
    part[threadIdx.y][threadIdx.x] = t;
    __syncthreads();
    if (threadIdx.y == 0 && col < D) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 16; ++w) v += part[w][threadIdx.x];
        out[col] = from_f32<W>(v);
    }
}

// ---------------------------------------------------------------- host side

// Packs a thread holds at most: the two sums of a pack's columns take 16 registers
// (fp32: 8), and 384 threads have 168 each (11136 x 3584 bf16: 64 us with 512 threads and
// spills, 55.5 with 384, 60.6 with 256; 768 threads of 2 packs: 68.7).  Widest row, by registers
// and shared memory: 24 KB, that is 12288 columns of 16 bits.
constexpr int kBwdPacks = 4;
constexpr int64_t kBwdRowBytes = kBwdThreads * kBwdPacks * 16;

size_t row_smem(const NormPlan& p, int tensors) { return (size_t)kStages * tensors * p.nv * p.threads() * 16; }
// `width`: columns of a row's packs; EDGE rows have gamma once a group.
size_t bwd_smem(const NormPlan& p, int64_t width, bool skip, bool edge) {
    const size_t rows = row_smem(p, skip ? 3 : 2), sums = (size_t)p.groups * 2 * padded((int)width) * 4;
    return (size_t)p.groups * 4 * kRed * 4 + (size_t)(edge ? p.groups : 1) * padded((int)width) * 4 + (rows > sums ? rows : sums);
}

// Backward: one CTA on each SM, of as many groups as threads, named barriers and shared
// memory allow, but one row for each SM before two for one.
NormPlan bwd_plan(int64_t M, int64_t width, int size, bool skip, bool edge) {
    NormPlan p = norm_plan(width, size, kBwdPacks, kBwdThreads);
    if (p.groups > 15) p.groups = 15;                      // barriers 1 .. 15
    const int64_t spread = (M + kPlanSms - 1) / kPlanSms;
    if (spread < p.groups) p.groups = spread > 0 ? (int)spread : 1;
    while (p.groups > 1 && bwd_smem(p, width, skip, edge) > kSmem) --p.groups;
    return p;
}
int bwd_ctas(int64_t M, const NormPlan& p) {
    const int64_t want = (M + p.groups - 1) / p.groups;
    return (int)(want < kPlanSms ? want : kPlanSms);
}

int64_t narrow_workers(int64_t M, int64_t D) {
    const int64_t most = kPlanSms * (int64_t)(narrow_threads(D) == 32 ? 16 : narrow_threads(D) == 128 ? 4 : 1);
    return M < most ? M : most;
}

int64_t wide_row_ranges(int64_t M, int64_t D, int vec) {
    const int64_t blocks = (D + 256 * vec - 1) / (256 * vec);
    int64_t r = (kPlanSms * 8 + blocks - 1) / blocks;
    if (r > 65535) r = 65535;
    return r < M ? r : M;
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

struct LaunchBwd {
    const NormBwd& a;
    const NormPlan& p;
    Lie lie;
    bool two_passes, packs;                // wide rows; they and gamma on 16-byte boundaries
    float2* sums;
    int planes;
    cudaStream_t s;
    template <class T, int NV, bool SKIP, bool EDGE>
    cudaError_t go() const {
        auto kern = layer_norm_bwd_kernel<T, NV, SKIP, EDGE>;
        const size_t smem = bwd_smem(p, reach(a.D, (int)sizeof(T), EDGE), SKIP, EDGE);
        cudaError_t e = allow_smem(kern, smem);
        if (e != cudaSuccess) return e;
        kern<<<(unsigned)planes, p.threads(), smem, s>>>(a);
        return cudaGetLastError();
    }
    template <class T, int NV>
    cudaError_t res() const {
        if (lie == kEdge) return a.skip ? go<T, NV, true, true>() : go<T, NV, false, true>();
        return a.skip ? go<T, NV, true, false>() : go<T, NV, false, false>();
    }
    template <class T, int THREADS>
    cudaError_t narrow() const {
        constexpr int rows = THREADS == 32 ? 4 : 1;
        auto kern = a.skip ? layer_norm_bwd_narrow_kernel<T, true, THREADS> : layer_norm_bwd_narrow_kernel<T, false, THREADS>;
        const size_t smem = (size_t)rows * 2 * (a.skip ? 3 : 2) * narrow_pitch(a.D * (int)sizeof(T));
        cudaError_t e = allow_smem(kern, smem);
        if (e != cudaSuccess) return e;
        kern<<<(unsigned)(planes / rows), THREADS * rows, smem, s>>>(a);
        return cudaGetLastError();
    }
    template <class T, int VEC>
    cudaError_t wide() const {
        const int64_t grid = a.M < kPlanSms * 4 ? a.M : kPlanSms * 4;
        layer_norm_bwd_wide_sums_kernel<T, VEC><<<(unsigned)grid, kMaxThreads, 0, s>>>(a, sums);
        const dim3 tiles((unsigned)((a.D + 256 * VEC - 1) / (256 * VEC)), (unsigned)planes);
        layer_norm_bwd_wide_kernel<T, VEC><<<tiles, 256, 0, s>>>(a, sums);
        return cudaGetLastError();
    }
    template <class T>
    cudaError_t run() const {
        if (two_passes) return packs ? wide<T, kVec<T>>() : wide<T, 1>();
        if (lie == kApart) {
            const int n = narrow_threads(a.D);
            return n == 32 ? narrow<T, 32>() : n == 128 ? narrow<T, 128>() : narrow<T, 512>();
        }
        return p.nv == 1 ? res<T, 1>() : p.nv == 2 ? res<T, 2>() : p.nv == 3 ? res<T, 3>() : res<T, 4>();
    }
};

}  // namespace
}  // namespace swiglu

using namespace swiglu;

extern "C" {

size_t swiglu_mlp_layer_norm_bwd_workspace_size(int64_t M, int64_t D) {
    if (M <= 0 || D <= 0) return 0;
    // whatever the type and the alignment: the most planes of the forms that take rows of this
    // width (the two-pass form: row sums too, and the widest packs have the most row ranges)
    int64_t planes = M < kPlanSms ? M : kPlanSms;
    if (D <= kNarrowWidth && (narrow_workers(M, D) + 3) / 4 * 4 > planes) planes = (narrow_workers(M, D) + 3) / 4 * 4;
    size_t sums = 0;
    if (D * 4 > kBwdRowBytes) {
        sums = round256((size_t)M * sizeof(float2));
        if (wide_row_ranges(M, D, 8) > planes) planes = wide_row_ranges(M, D, 8);
    }
    return sums + 2 * round256((size_t)planes * D * 4);
}

swiglu_status swiglu_mlp_layer_norm_bwd(const void* dy, int64_t lddy, const void* s, int64_t lds, const void* gamma,
                                        const float* mean, const float* rstd, const void* dskip, int64_t ldskip,
                                        void* dx, int64_t lddx, void* dgamma, void* dbeta, int64_t M, int64_t D,
                                        int type, int param_type, void* workspace, size_t workspace_bytes,
                                        void* stream) {
    swiglu_status rc = norm_check(M, D, type, param_type);
    if (rc != SWIGLU_OK) return rc;
    const size_t n = type_bytes(type), np = type_bytes(param_type);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    int sms;
    if (misaligned(dgamma, np) || misaligned(dbeta, np))
        return fail(SWIGLU_ERR_MISALIGNED, "layer norm: a pointer is not aligned to its element");
    if (M == 0) {
        rc = device_sms(&sms);
        if (rc != SWIGLU_OK) return rc;
        for (void* p : {dgamma, dbeta}) {
            cudaError_t e = p ? cudaMemsetAsync(p, 0, (size_t)D * np, st) : cudaSuccess;
            if (e != cudaSuccess) return fail(SWIGLU_ERR_CUDA, "cudaMemsetAsync(parameter gradients)", e);
        }
        return SWIGLU_OK;
    }
    if (!dy || !s || !mean || !rstd || !dx || !workspace)
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a required pointer is null");
    if (lddy < D || lds < D || lddx < D || (dskip && ldskip < D))
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a row stride is smaller than the width");
    if (misaligned(dy, n) || misaligned(s, n) || misaligned(dskip, n) || misaligned(dx, n) || misaligned(gamma, np) ||
        misaligned(mean, 4) || misaligned(rstd, 4) || !aligned16(workspace))
        return fail(SWIGLU_ERR_MISALIGNED, "layer norm: a pointer is not aligned to its element, or the workspace to 16 bytes");
    if (workspace_bytes < swiglu_mlp_layer_norm_bwd_workspace_size(M, D))
        return fail(SWIGLU_ERR_WORKSPACE_TOO_SMALL, "layer norm: workspace smaller than the size query returns");
    rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    Rows16 v{(int)n};
    v.add(dy, lddy), v.add(s, lds), v.add(dskip, ldskip), v.add(dx, lddx);
    Lie lie = v.lie(D);
    // Shifted packs pay where a group has rows to spread their gamma and column sums over (element
    // by element, then packs, us: bf16 3000 x 5003 51, 31; 40000 x 65 31, 28; fp32 40000 x 33 28, 21;
    // but one row for each SM, 152 x 5003: 10.8, 13.9), and up to the widest row they take.
    if (lie == kEdge && ((M <= kPlanSms && D <= kNarrowWidth) || reach(D, (int)n, true) * (int64_t)n > kBwdRowBytes)) lie = kApart;
    const bool wide = lie == kApart ? D > kNarrowWidth : D * (int64_t)n > kBwdRowBytes;
    const bool packs = lie == kWhole && !misaligned(gamma, 16), edge = lie == kEdge;
    const NormPlan p = bwd_plan(M, reach(D, (int)n, edge), (int)n, dskip != nullptr, edge);
    // a worker of one warp comes with three others
    const int planes = (int)(wide            ? wide_row_ranges(M, D, packs ? 16 / (int)n : 1)
                             : lie == kApart ? narrow_threads(D) == 32 ? (narrow_workers(M, D) + 3) / 4 * 4 : narrow_workers(M, D)
                                             : bwd_ctas(M, p));
    uint8_t* w = static_cast<uint8_t*>(workspace);
    float2* sums = reinterpret_cast<float2*>(w);
    if (wide) w += round256((size_t)M * sizeof(float2));
    float* pg = reinterpret_cast<float*>(w);
    float* pb = reinterpret_cast<float*>(w + round256((size_t)planes * D * 4));
    const NormBwd a{dy, s, gamma, dskip, mean, rstd, dx, dgamma ? pg : nullptr, dbeta ? pb : nullptr,
                    lddy, lds, ldskip, lddx, M, (int)D, p.lanes, param_type == SWIGLU_FP32};
    rc = launch_traced(SWIGLU_KERNEL_NORM_BWD, st,
                       [&] { return with_type(type, LaunchBwd{a, p, lie, wide, packs, sums, planes, st}); });
    if (rc != SWIGLU_OK || (!dgamma && !dbeta)) return rc;
    return launch_traced(SWIGLU_KERNEL_NORM_PARAMS, st, [&] {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cfg.gridDim = dim3((unsigned)((D + 31) / 32), 2);
        cfg.blockDim = dim3(32, 16);
        cfg.stream = st;
        const float *g = pg, *b = pb;
        const int d = (int)D;
        if (param_type == SWIGLU_FP32)
            return cudaLaunchKernelEx(&cfg, layer_norm_params_kernel<float>, g, b, (float*)dgamma, (float*)dbeta, planes, d);
        if (param_type == SWIGLU_FP16)
            return cudaLaunchKernelEx(&cfg, layer_norm_params_kernel<__half>, g, b, (__half*)dgamma, (__half*)dbeta, planes, d);
        return cudaLaunchKernelEx(&cfg, layer_norm_params_kernel<__nv_bfloat16>, g, b, (__nv_bfloat16*)dgamma,
                                  (__nv_bfloat16*)dbeta, planes, d);
    });
}

}  // extern "C"
