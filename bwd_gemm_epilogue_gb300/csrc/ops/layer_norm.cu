// layer_norm.cu -- layer norm forward and backward (include/swiglu_ops.h).
//
// Both directions are bound by HBM: a row is read once into registers, its statistics are
// reduced there, and the result is written once.  At the HBM rate an SM has about 40
// instructions a column for all of it, so what a row costs besides its columns has to be
// spread over many of them, and the columns' arithmetic runs in packed pairs: a row belongs
// to a group of `lanes` threads with NV packs of 16 bytes each (pack k = q * lanes + lane of
// the row, q < NV), and a group walks its own rows, with the next two in flight to shared
// memory (registers could hold one, and its latency showed: 92 us backward instead of
// the ring's for 11136 x 3584 bf16).
//
// Rows that do not start on 16-byte boundaries (odd widths, strides, bases) move in aligned
// 16-byte pieces all the same: each lane copies the aligned piece its pack starts in, takes
// the rest from its neighbour's and shifts the two together; stores likewise, with single
// elements at the ends of a warp's span.
#include "../host.h"
#include "convert.cuh"
#include "swiglu_ops.h"

namespace swiglu {
namespace {

constexpr int kPlanSms = 152;      // grids are planned for the GB300, so that the workspace query sees no device
constexpr int kMaxThreads = 512;   // the forms for rows too wide for registers
constexpr int kBwdThreads = 512;

struct NormFwd {
    const void *x, *r, *gamma, *beta;
    void *y, *s;
    float *mean, *rstd;
    int64_t ldx, ldr, ldy, lds, M;
    int D, lanes, gf32;
    float eps;
};

struct NormBwd {
    const void *dy, *s, *gamma, *skip;
    const float *mean, *rstd;
    void* dx;
    float *pg, *pb;                // partial planes [gridDim][D] of dgamma and dbeta (NULL: not wanted)
    int64_t lddy, lds, ldk, lddx, M;
    int D, lanes, gf32;
};

// ---------------------------------------------------------------- 16-byte packs of a row

template <class T>
constexpr int kVec = 16 / (int)sizeof(T);

// The first `n` elements of a partial pack, the others zero.
template <class T>
__device__ __forceinline__ void keep_first(F2* v, int n) {
#pragma unroll
    for (int i = 0; i < kVec<T> / 2; ++i) {
        const float2 f = split(v[i]);
        v[i] = f2(2 * i < n ? f.x : 0.f, 2 * i + 1 < n ? f.y : 0.f);
    }
}

// 16 bytes from byte s (0 < s < 16, a multiple of the element) of the 32 bytes a, b.
__device__ __forceinline__ uint4 shift_bytes(const uint4& a, const uint4& b, int s) {
    uint32_t c[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const bool two = s & 8, one = s & 4;
#pragma unroll
    for (int i = 0; i < 6; ++i) c[i] = two ? c[i + 2] : c[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) c[i] = one ? c[i + 1] : c[i];
    const int bits = (s & 2) * 8;
    return make_uint4(__funnelshift_r(c[0], c[1], bits), __funnelshift_r(c[1], c[2], bits),
                      __funnelshift_r(c[2], c[3], bits), __funnelshift_r(c[3], c[4], bits));
}

// The aligned 16 bytes at p, of which only [lo, hi) may be read; what lies outside is zero.
template <class T>
__device__ __noinline__ uint4 load_edge(uintptr_t p, uintptr_t lo, uintptr_t hi) {
    uint32_t u[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) {
        const uintptr_t at = p + i * sizeof(T);
        if (at >= lo && at < hi) {
            if constexpr (sizeof(T) == 4) u[i] = *reinterpret_cast<const uint32_t*>(at);
            else u[i / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(at) << (i % 2 * 16);
        }
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ void copy_async(uint32_t dst, uintptr_t src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ uint4 load_smem(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void store_smem(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void commit_async() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void wait_async() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A row read and the next one in flight, in shared memory, filled by asynchronous copies.  A
// thread copies and reads its own packs, so this needs no barrier; of an unaligned row it
// copies the aligned pieces its packs start in, and finds the next piece in its neighbour's
// slot (the last lane of a warp copies one piece more).  Layout: [stage][pack][slot].
constexpr int kStages = 2;

__host__ __device__ constexpr int ring_slots(int threads) { return threads / 32 * 33; }

// One tensor's share of the ring, and the group's next row of it.
template <class T, int NV, bool SHIFT>
struct Rows {
    const char *next = nullptr, *now = nullptr;   // this lane's pack 0 of the row to copy; of the row to read
    int64_t hop = 0;                       // bytes from a group's row to its next
    uint32_t slot;                         // shared address of this thread's slot, stage 0, pack 0
    uint32_t per;                          // bytes from a pack's slots to the next pack's
    uintptr_t lo, hi;                      // SHIFT: the tensor's bytes
    __device__ __forceinline__ void init(const T* base, int64_t ld, int64_t row, int64_t step, int lane, int64_t M,
                                         int D, uint32_t smem, int tensor) {
        next = now = reinterpret_cast<const char*>(base + row * ld) + lane * 16;
        hop = step * ld * (int64_t)sizeof(T);
        per = ring_slots(blockDim.x) * 16;
        slot = smem + tensor * kStages * NV * per + (threadIdx.x / 32 * 33 + threadIdx.x % 32) * 16;
        lo = reinterpret_cast<uintptr_t>(base);
        hi = lo + (uintptr_t)((M - 1) * ld + D) * sizeof(T);
    }
    // Copies the group's next row into a stage; `lane16`: 16 x lane, `pitch`: 16 x lanes.
    __device__ __forceinline__ void issue(int stage, int lane16, int pitch, int row_bytes) {
        const uint32_t to = slot + stage * NV * per;
        if constexpr (!SHIFT) {
#pragma unroll
            for (int q = 0; q < NV; ++q)
                if (q < NV - 1 || q * pitch + lane16 < row_bytes)
                    copy_async(to + q * per, reinterpret_cast<uintptr_t>(next) + q * pitch, 16);
        } else {
            const int m = (int)(reinterpret_cast<uintptr_t>(next) & 15);
            auto piece = [&](int at, uint32_t dst) {       // the aligned piece at byte `at` - m of the row
                if (at - m >= row_bytes) return;
                const uintptr_t p = reinterpret_cast<uintptr_t>(next) - lane16 + at - m;
                if (p >= lo) copy_async(dst, p, p + 16 <= hi ? 16 : (int)(hi - p));
                else store_smem(dst, load_edge<T>(p, lo, hi));
            };
#pragma unroll
            for (int q = 0; q < NV; ++q) {
                piece(q * pitch + lane16, to + q * per);
                if ((threadIdx.x & 31) == 31) piece(q * pitch + lane16 + 16, to + q * per + 16);
            }
        }
        next += hop;
    }
    // Pack q of the row to read, once its copies have landed.
    __device__ __forceinline__ uint4 get(int stage, int q) const {
        const uint32_t from = slot + (stage * NV + q) * per;
        const uint4 a = load_smem(from);
        if constexpr (SHIFT) {
            const int m = (int)(reinterpret_cast<uintptr_t>(now) & 15);
            if (m) return shift_bytes(a, load_smem(from + 16), m);
        }
        return a;
    }
    __device__ __forceinline__ void advance() {
        if (SHIFT) now += hop;
    }
};

// Stores pack k, of which `n` elements (0 .. VEC) are the row's: an aligned piece is stored
// by the lane whose pack it ends in where both its parts are the row's and the warp's, all
// else element by element.
template <class T>
__device__ __forceinline__ void store_shifted(T* row, int k, int n, const uint4& v) {
    constexpr int V = kVec<T>;
    T* p = row + (int64_t)k * V;
    const int m = (int)(reinterpret_cast<uintptr_t>(row) & 15), lane = threadIdx.x & 31;
    const int split_at = (16 - m) / (int)sizeof(T);        // elements of the pack before the aligned boundary
    uint4 prev;
    prev.x = __shfl_up_sync(0xffffffffu, v.x, 1);
    prev.y = __shfl_up_sync(0xffffffffu, v.y, 1);
    prev.z = __shfl_up_sync(0xffffffffu, v.z, 1);
    prev.w = __shfl_up_sync(0xffffffffu, v.w, 1);
    const bool piece = n >= split_at && (m == 0 || lane > 0);
    bool next = __shfl_down_sync(0xffffffffu, piece, 1);
    if (lane == 31) next = false;
    if (piece) *reinterpret_cast<uint4*>(reinterpret_cast<uintptr_t>(p) - m) = m == 0 ? v : shift_bytes(prev, v, 16 - m);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        if (i < n && (i < split_at ? !piece : !next)) {
            if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(p)[i] = u[i];
            else reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(u[i / 2] >> (i % 2 * 16));
        }
    }
}

// gamma or beta as fp32 in shared memory: the first 16 bytes of every pack's values, then
// (16-bit rows) the second 16 bytes of every pack's, so that a warp's 16-byte reads touch
// every bank once.
__host__ __device__ constexpr int padded(int D) { return (D + 7) / 8 * 8; }

template <class T>
__device__ __forceinline__ void stage_param(float* to, const void* p, int gf32, int D, float none) {
    const int half = padded(D) / 2;
    auto put = [&](int c, float v) { to[sizeof(T) == 4 ? c : (c & 4 ? half : 0) + (c >> 3) * 4 + (c & 3)] = v; };
    if (gf32 && (reinterpret_cast<uintptr_t>(p) & 15) == 0 && p != nullptr && D % 4 == 0) {
#pragma unroll 4
        for (int c = threadIdx.x * 4; c < D; c += blockDim.x * 4) {
            const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const float*>(p) + c);
            *reinterpret_cast<uint4*>(&to[sizeof(T) == 4 ? c : (c & 4 ? half : 0) + (c >> 3) * 4]) = v;
        }
        for (int c = D + threadIdx.x; c < padded(D); c += blockDim.x) put(c, 0.f);
        return;
    }
#pragma unroll 8
    for (int c = threadIdx.x; c < padded(D); c += blockDim.x)
        put(c, c >= D ? 0.f : p == nullptr ? none : gf32 ? static_cast<const float*>(p)[c] : to_f32(static_cast<const T*>(p)[c]));
}

// Pack k of one, as pairs.
template <class T>
__device__ __forceinline__ void load_staged(F2* o, uint32_t p, int k, int D) {
    unpack16<float>(load_smem(p + k * 16), o);
    if constexpr (sizeof(T) == 2) unpack16<float>(load_smem(p + padded(D) * 2 + k * 16), o + 2);
}

// The same from global memory (`n` elements are the row's; !SHIFT: whole packs, aligned).
template <class T, bool SHIFT>
__device__ __forceinline__ void load_param16(F2* o, const void* p, int gf32, int k, int n, float none) {
    constexpr int V = kVec<T>;
    const bool whole = !SHIFT || (n == V && (reinterpret_cast<uintptr_t>(p) & 15) == 0);
    if (p == nullptr) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) o[i] = f2(none);
    } else if (!whole) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            float f[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int at = k * V + 2 * i + j;
                f[j] = 2 * i + j >= n ? 0.f : gf32 ? static_cast<const float*>(p)[at] : to_f32(static_cast<const T*>(p)[at]);
            }
            o[i] = f2(f[0], f[1]);
        }
    } else if (sizeof(T) == 2 && gf32) {
        const uint4* q = reinterpret_cast<const uint4*>(p) + 2 * k;
        unpack16<float>(q[0], o);
        unpack16<float>(q[1], o + 2);
    } else {
        unpack16<T>(reinterpret_cast<const uint4*>(p)[k], o);
    }
}

// ---------------------------------------------------------------- sums over a row

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Barrier of a group of threads (barrier 0 is __syncthreads').
__device__ __forceinline__ void group_sync(int group, int lanes) {
    asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");
}

// Sums over the group's `lanes` threads.  One warp: shuffles.  More: shuffles, then every
// thread adds the warps' sums from shared memory in warp order.  `red`: kRed entries for each
// of two buffers, which the caller alternates, so that one barrier a reduction is enough: a
// buffer is rewritten only after the other one's barrier, which every reader of the first
// has passed.  The entries past the group's warps hold zeros.
constexpr int kRed = 24;

__device__ __forceinline__ float row_sum(float v, int group, int lanes, float* red, int buf) {
    v = warp_sum(v);
    if (lanes == 32) return v;
    red += buf * kRed;
    if ((threadIdx.x & 31) == 0) red[(threadIdx.x - group * lanes) >> 5] = v;
    group_sync(group, lanes);
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kRed; w += 4) {
        if (w * 32 >= lanes) break;
        const float4 f = *reinterpret_cast<const float4*>(red + w);
        v += (f.x + f.y) + (f.z + f.w);
    }
    return v;
}

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

// ---------------------------------------------------------------- forward

// What of pack k = q * lanes + lane is the row's: the plan gives a row ceil(packs / lanes)
// packs a thread, so only the last one can end past it.
template <class T, int NV, bool SHIFT>
__device__ __forceinline__ int pack_elements(int q, int k, int D) {
    constexpr int V = kVec<T>;
    if (q < NV - 1 && !SHIFT) return V;
    const int left = D - k * V;
    return left >= V ? V : left > 0 ? left : 0;
}

// The packs of an unaligned row that a warp holds, as the aligned pieces they start in: lane
// l's of pack q, and in lane q the piece that follows pack q of the last lane.
template <class T, int NV>
struct Pieces {
    uint4 a[NV], after;
    int m;                                 // bytes of the first piece before the row
    __device__ __forceinline__ void load(const T* row, int lane16, int pitch, int row_bytes, uintptr_t lo, uintptr_t hi) {
        const uintptr_t start = reinterpret_cast<uintptr_t>(row);
        const int l = threadIdx.x & 31;
        m = (int)(start & 15);
        auto piece = [&](int at) {
            const uintptr_t p = start - m + at;
            if (at - m >= row_bytes) return make_uint4(0, 0, 0, 0);
            if (p >= lo && p + 16 <= hi) return *reinterpret_cast<const uint4*>(p);
            return load_edge<T>(p, lo, hi);
        };
#pragma unroll
        for (int q = 0; q < NV; ++q) a[q] = piece(q * pitch + lane16);
        after = l < NV ? piece(l * pitch + lane16 - l * 16 + 512) : make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ uint4 pack(int q) const {
        if (m == 0) return a[q];
        uint4 b;
        const bool last = (threadIdx.x & 31) == 31;
        const uint32_t own[4] = {a[q].x, a[q].y, a[q].z, a[q].w}, end[4] = {after.x, after.y, after.z, after.w};
        uint32_t next[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t n = __shfl_down_sync(0xffffffffu, own[i], 1), e = __shfl_sync(0xffffffffu, end[i], q);
            next[i] = last ? e : n;
        }
        b = make_uint4(next[0], next[1], next[2], next[3]);
        return shift_bytes(a[q], b, m);
    }
};

// One row for each group of `lanes` threads: a CTA is one row of more than a warp, or four
// rows of one.  Many small CTAs take turns at loading, reducing and storing; a persistent
// form with the next row in flight in shared memory took 57 us where this takes 53
// (11136 x 3584 bf16).  The statistics need one barrier: a warp centres its columns on its
// own mean, and the warps' (mean, sum of squares about it) are joined exactly.
template <class T, int NV, bool SHIFT, bool RES, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) layer_norm_fwd_kernel(const NormFwd a) {
    constexpr int V = kVec<T>, P = V / 2;
    __shared__ float2 red[THREADS / 32];
    const int lanes = a.lanes, lane = threadIdx.x % lanes, D = a.D;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / lanes) + threadIdx.x / lanes;
    if (row >= a.M) return;                // whole warps; with more than one warp a row, no thread
    const int lane16 = lane * 16, pitch = lanes * 16, row_bytes = D * (int)sizeof(T);
    const T* x = static_cast<const T*>(a.x) + row * a.ldx;
    const T* r = static_cast<const T*>(a.r) + row * a.ldr;
    F2 v[NV * P];
    if constexpr (SHIFT) {
        const uintptr_t x0 = reinterpret_cast<uintptr_t>(a.x), r0 = reinterpret_cast<uintptr_t>(a.r);
        Pieces<T, NV> px, pr;
        px.load(x, lane16, pitch, row_bytes, x0, x0 + ((a.M - 1) * a.ldx + D) * sizeof(T));
        if (RES) pr.load(r, lane16, pitch, row_bytes, r0, r0 + ((a.M - 1) * a.ldr + D) * sizeof(T));
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int n = pack_elements<T, NV, SHIFT>(q, q * lanes + lane, D);
            F2* w = v + q * P;
            unpack16<T>(px.pack(q), w);
            if (RES) {
                F2 f[P];
                unpack16<T>(pr.pack(q), f);
#pragma unroll
                for (int i = 0; i < P; ++i) w[i] = w[i] + f[i];
            }
            if (n < V) keep_first<T>(w, n);
        }
    } else {
        uint4 px[NV], pr[NV];
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int k = q * lanes + lane;
            px[q] = pr[q] = make_uint4(0, 0, 0, 0);
            if (pack_elements<T, NV, SHIFT>(q, k, D)) {
                px[q] = __ldcs(reinterpret_cast<const uint4*>(x) + k);
                if (RES) pr[q] = __ldcs(reinterpret_cast<const uint4*>(r) + k);
            }
        }
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            F2* w = v + q * P;
            unpack16<T>(px[q], w);
            if (RES) {
                F2 f[P];
                unpack16<T>(pr[q], f);
#pragma unroll
                for (int i = 0; i < P; ++i) w[i] = w[i] + f[i];
            }
        }
    }
    if (RES) {
        T* si = static_cast<T*>(a.s) + row * a.lds;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int k = q * lanes + lane, n = pack_elements<T, NV, SHIFT>(q, k, D);
            const uint4 o = pack16<T>(v + q * P);
            if (SHIFT) store_shifted<T>(si, k, n, o);
            else if (n) reinterpret_cast<uint4*>(si)[k] = o;
        }
    }
    F2 sum2 = f2(0.f);
#pragma unroll
    for (int i = 0; i < NV * P; ++i) sum2 = sum2 + v[i];
    // columns of warp w: of every pack its 32 * V from (q * lanes + 32 w) * V
    auto columns = [&](int w) {
        int n = 0;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int left = D - (q * lanes + 32 * w) * V;
            n += left >= 32 * V ? 32 * V : left > 0 ? left : 0;
        }
        return (float)n;
    };
    const float2 ss = split(sum2);
    const int warp = (threadIdx.x % lanes) >> 5, warps = lanes >> 5;
    const float mine = columns(warp);
    float mean = warp_sum(ss.x + ss.y) / fmaxf(mine, 1.f);
    const F2 mu = f2(-mean);
    F2 sq2 = f2(0.f);
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        const int n = pack_elements<T, NV, SHIFT>(q, q * lanes + lane, D);
        if (n > 0) {
            F2 c[P];
#pragma unroll
            for (int i = 0; i < P; ++i) c[i] = v[q * P + i] + mu;
            if (SHIFT && n < V) keep_first<T>(c, n);
#pragma unroll
            for (int i = 0; i < P; ++i) sq2 = fma(c[i], c[i], sq2);
        }
    }
    const float2 qq = split(sq2);
    float sq = warp_sum(qq.x + qq.y);
    if (warps > 1) {
        if ((threadIdx.x & 31) == 0) red[warp] = make_float2(mean, sq);
        __syncthreads();
        float total = 0.f;
        for (int w = 0; w < warps; ++w) total += columns(w) * red[w].x;
        mean = total / (float)D;
        sq = 0.f;
        for (int w = 0; w < warps; ++w) {
            const float d = red[w].x - mean;
            sq += red[w].y + columns(w) * d * d;
        }
    }
    const float rstd = __frsqrt_rn(sq / (float)D + a.eps);
    const F2 rs = f2(rstd), m2 = f2(-mean);
    T* yi = static_cast<T*>(a.y) + row * a.ldy;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        const int k = q * lanes + lane, n = pack_elements<T, NV, SHIFT>(q, k, D);
        uint4 o = make_uint4(0, 0, 0, 0);
        if (n > 0) {
            F2 g[P], b[P];
            load_param16<T, SHIFT>(g, a.gamma, a.gf32, k, n, 1.f);
            load_param16<T, SHIFT>(b, a.beta, a.gf32, k, n, 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i) g[i] = fma((v[q * P + i] + m2) * rs, g[i], b[i]);
            o = pack16<T>(g);
            if (!SHIFT) __stcs(reinterpret_cast<uint4*>(yi) + k, o);
        }
        if (SHIFT) store_shifted<T>(yi, k, n, o);
    }
    if (lane == 0 && a.mean) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
}

// gamma or beta at column `col`, in the row's type or in fp32 (the forms for wide rows).
template <class T, int VEC>
__device__ __forceinline__ void load_param(float* o, const void* p, int gf32, int col, float none) {
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[j] = none;
    } else if (gf32) {
        constexpr int V4 = VEC >= 4 ? 4 : 1;
#pragma unroll
        for (int q = 0; q < VEC / V4; ++q)
            load_pack<float, V4>(static_cast<const float*>(p) + col + q * V4).unpack(o + q * V4);
    } else {
        load_pack<T, VEC>(static_cast<const T*>(p) + col).unpack(o);
    }
}

// A row wider than the registers hold: three passes over it, the last two from L2.
template <class T, int VEC>
__global__ void __launch_bounds__(kMaxThreads) layer_norm_fwd_wide_kernel(const NormFwd a) {
    __shared__ __align__(16) float red[2 * kRed];
    if (threadIdx.x < 2 * kRed) red[threadIdx.x] = 0.f;
    __syncthreads();
    const float inv = 1.f / (float)a.D;
    for (int64_t row = blockIdx.x; row < a.M; row += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + row * a.ldx;
        const T* r = a.r ? static_cast<const T*>(a.r) + row * a.ldr : nullptr;
        auto load = [&](int col, float* v) {
            load_pack<T, VEC>(x + col).unpack(v);
            if (r) {
                float e[VEC];
                load_pack<T, VEC>(r + col).unpack(e);
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[j] += e[j];
            }
        };
        const int first = threadIdx.x * VEC, hop = blockDim.x * VEC;
        float v[VEC], sum = 0.f, sq = 0.f;
        for (int64_t c = first; c < a.D; c += hop) {
            load((int)c, v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sum += v[j];
            if (r) store_pack<T, VEC>(static_cast<T*>(a.s) + row * a.lds + c, v);
        }
        const float mean = row_sum(sum, 0, blockDim.x, red, 0) * inv;
        for (int64_t c = first; c < a.D; c += hop) {
            load((int)c, v);
#pragma unroll
            for (int j = 0; j < VEC; ++j) sq += (v[j] - mean) * (v[j] - mean);
        }
        const float rstd = __frsqrt_rn(row_sum(sq, 0, blockDim.x, red, 1) * inv + a.eps);
        for (int64_t c = first; c < a.D; c += hop) {
            float g[VEC], b[VEC];
            load((int)c, v);
            load_param<T, VEC>(g, a.gamma, a.gf32, (int)c, 1.f);
            load_param<T, VEC>(b, a.beta, a.gf32, (int)c, 0.f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) v[j] = (v[j] - mean) * rstd * g[j] + b[j];
            store_pack<T, VEC>(static_cast<T*>(a.y) + row * a.ldy + c, v);
        }
        if (threadIdx.x == 0 && a.mean) {
            a.mean[row] = mean;
            a.rstd[row] = rstd;
        }
    }
}

// ---------------------------------------------------------------- backward

// The row's two sums, dx, and fp32 column sums of dy * xh and dy over the group's rows, kept
// in registers; the CTA's groups are added in shared memory at the end and written once, as
// this CTA's partial planes.  A row is read from the ring twice, before and after the
// reduction, which costs less than keeping xh and g beside the column sums.  xh = s * rstd - mean * rstd, and
// dx = g * rstd + s * A + B with A = -c2 * rstd^2, B = c2 * mean * rstd^2 - c1 * rstd.
// Shared memory: red [groups][2][kRed] pairs, gamma (whole packs, fp32), then the rows in
// flight, and after them the groups' column sums in their place.
template <class T, int NV, bool SHIFT, bool SKIP>
__global__ void __launch_bounds__(kBwdThreads) layer_norm_bwd_kernel(const NormBwd a) {
    constexpr int V = kVec<T>, P = V / 2;
    extern __shared__ uint4 smem[];
    const int lanes = a.lanes, lane = threadIdx.x % lanes, group = threadIdx.x / lanes, D = a.D;
    const int rows = blockDim.x / lanes;
    float2* red = reinterpret_cast<float2*>(smem) + group * 2 * kRed;
    float* gamma = reinterpret_cast<float*>(smem) + rows * 4 * kRed;
    float* acc = gamma + padded(D);
    const int64_t step = (int64_t)gridDim.x * rows;
    int64_t row = (int64_t)blockIdx.x * rows + group;
    const int lane16 = lane * 16, pitch = lanes * 16, row_bytes = D * (int)sizeof(T);
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(acc);
    Rows<T, NV, SHIFT> dy, s, skip;
    dy.init(static_cast<const T*>(a.dy), a.lddy, row, step, lane, a.M, D, ring, 0);
    s.init(static_cast<const T*>(a.s), a.lds, row, step, lane, a.M, D, ring, 1);
    if (SKIP) skip.init(static_cast<const T*>(a.skip), a.ldk, row, step, lane, a.M, D, ring, 2);
    auto issue = [&](int stage, int64_t i) {
        if (i < a.M) {
            dy.issue(stage, lane16, pitch, row_bytes);
            s.issue(stage, lane16, pitch, row_bytes);
            if (SKIP) skip.issue(stage, lane16, pitch, row_bytes);
        }
        commit_async();
    };
    cudaTriggerProgrammaticLaunchCompletion();             // the parameters' kernel may come up meanwhile
    issue(0, row);
    for (int i = threadIdx.x; i < rows * 4 * kRed; i += blockDim.x) reinterpret_cast<float*>(smem)[i] = 0.f;
    stage_param<T>(gamma, a.gamma, a.gf32, D, 1.f);
    const uint32_t gamma_at = (uint32_t)__cvta_generic_to_shared(gamma);
    __syncthreads();
    F2 dg[NV * P], db[NV * P];
#pragma unroll
    for (int i = 0; i < NV * P; ++i) dg[i] = db[i] = f2(0.f);
    float mean = 0.f, rstd = 0.f;
    if (row < a.M) mean = a.mean[row], rstd = a.rstd[row];
    const float inv = 1.f / (float)D;
    for (int stage = 0; row < a.M; row += step, stage ^= 1, dy.advance(), s.advance(), skip.advance()) {
        if (SHIFT) __syncwarp();           // the neighbours have read the stage that is filled next
        issue(stage ^ 1, row + step);
        const float mu = mean, rs = rstd;
        if (row + step < a.M) mean = a.mean[row + step], rstd = a.rstd[row + step];
        wait_async<1>();
        if (SHIFT) __syncwarp();
        const F2 rs2 = f2(rs), shift = f2(-mu * rs);
        F2 c1 = f2(0.f), c2 = f2(0.f);
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int k = q * lanes + lane, n = pack_elements<T, NV, SHIFT>(q, k, D);
            if (n > 0) {
                F2 w[P], d[P], xs[P];
                load_staged<T>(w, gamma_at, k, D);
                unpack16<T>(dy.get(stage, q), d);
                unpack16<T>(s.get(stage, q), xs);
                if (SHIFT && n < V) keep_first<T>(d, n), keep_first<T>(xs, n);
#pragma unroll
                for (int i = 0; i < P; ++i) {
                    const F2 xh = fma(xs[i], rs2, shift), g = d[i] * w[i];
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
        const F2 A = f2(-c.y * rs), B = f2(c.y * mu * rs - c.x);
        T* oi = static_cast<T*>(a.dx) + row * a.lddx;
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int k = q * lanes + lane, n = pack_elements<T, NV, SHIFT>(q, k, D);
            uint4 o = make_uint4(0, 0, 0, 0);
            if (n > 0) {
                F2 w[P], d[P], xs[P];
                load_staged<T>(w, gamma_at, k, D);
                unpack16<T>(dy.get(stage, q), d);
                unpack16<T>(s.get(stage, q), xs);
#pragma unroll
                for (int i = 0; i < P; ++i) w[i] = fma(d[i] * w[i], rs2, fma(xs[i], A, B));
                if (SKIP) {
                    unpack16<T>(skip.get(stage, q), d);
#pragma unroll
                    for (int i = 0; i < P; ++i) w[i] = w[i] + d[i];
                }
                o = pack16<T>(w);
                if (!SHIFT) reinterpret_cast<uint4*>(oi)[k] = o;
            }
            if (SHIFT) store_shifted<T>(oi, k, n, o);
        }
    }
    if (a.pg == nullptr && a.pb == nullptr) return;
    // the groups' sums meet in the ring's place: [group][2][columns, 16-byte pieces of packs apart]
    wait_async<0>();
    __syncthreads();
    const int width = padded(D), half = sizeof(T) == 2 ? width / 2 : 0;
    float* mine = acc + group * 2 * width;
#pragma unroll
    for (int q = 0; q < NV; ++q) {
        const int k = q * lanes + lane;
        if (pack_elements<T, NV, true>(q, k, D) > 0) {
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
    for (int c = threadIdx.x; c < D; c += blockDim.x) {
        const float* p = acc + (sizeof(T) == 4 ? c : (c & 4 ? half : 0) + (c >> 3) * 4 + (c & 3));
        float g = 0.f, b = 0.f;
        for (int w = 0; w < rows; ++w, p += 2 * width) g += p[0], b += p[width];
        if (a.pg) a.pg[(int64_t)blockIdx.x * D + c] = g;
        if (a.pb) a.pb[(int64_t)blockIdx.x * D + c] = b;
    }
}

// Rows wider than the registers hold, in two passes: the two sums of every row, then dx
// and the column sums of a block of columns over a range of rows.
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
        float2 c = make_float2(0.f, 0.f);
        for (int64_t col = threadIdx.x * VEC; col < a.D; col += blockDim.x * VEC) {
            float w[VEC], d[VEC], xs[VEC];
            load_pack<T, VEC>(dy + col).unpack(d);
            load_pack<T, VEC>(s + col).unpack(xs);
            load_param<T, VEC>(w, a.gamma, a.gf32, (int)col, 1.f);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float g = d[j] * w[j];
                c.x += g;
                c.y += g * ((xs[j] - mean) * rstd);
            }
        }
        c = row_sum2(c, 0, blockDim.x, red, buf);
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

// dgamma and dbeta: the planes added in plane order (16 strided runs, then the runs).
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

// How a launch covers its rows: `nv` packs a thread, `lanes` threads a row, `groups` rows a
// CTA at a time.
struct NormPlan {
    int nv, lanes, groups;
    int threads() const { return lanes * groups; }
};

// Packs a thread holds at most.  Backward: 16 columns (fp32: 8), whose two sums take 32
// registers.
constexpr int kFwdPacks = 4, kBwdPacks = 4;
constexpr size_t kSmem = 227 * 1024;

size_t row_smem(const NormPlan& p, int tensors) { return (size_t)kStages * tensors * p.nv * ring_slots(p.threads()) * 16; }
size_t bwd_smem(const NormPlan& p, int64_t D, bool skip) {
    const size_t rows = row_smem(p, skip ? 3 : 2), sums = (size_t)p.groups * 2 * padded((int)D) * 4;
    return (size_t)p.groups * 4 * kRed * 4 + (size_t)padded((int)D) * 4 + (rows > sums ? rows : sums);
}

NormPlan norm_plan(int64_t D, int size, int packs, int threads) {
    NormPlan p;
    const int64_t all = (D * size + 15) / 16;
    p.lanes = (int)((all + packs * 32 - 1) / (packs * 32) * 32);
    p.nv = (int)((all + p.lanes - 1) / p.lanes);
    p.groups = threads / p.lanes > 1 ? threads / p.lanes : 1;
    return p;
}

// Forward: CTAs of one row of more than a warp, or of four rows of one.
NormPlan fwd_plan(int64_t D, int size) {
    NormPlan p = norm_plan(D, size, kFwdPacks, 128);
    if (p.lanes > 32) p.groups = 1;
    return p;
}

// Backward: one CTA on each SM, of as many groups as threads, named barriers and shared
// memory allow, but one row for each SM before two for one.
NormPlan bwd_plan(int64_t M, int64_t D, int size, bool skip) {
    NormPlan p = norm_plan(D, size, kBwdPacks, kBwdThreads);
    if (p.groups > 15) p.groups = 15;                      // barriers 1 .. 15
    const int64_t spread = (M + kPlanSms - 1) / kPlanSms;
    if (spread < p.groups) p.groups = spread > 0 ? (int)spread : 1;
    while (p.groups > 1 && bwd_smem(p, D, skip) > kSmem) --p.groups;
    return p;
}
int bwd_ctas(int64_t M, const NormPlan& p) {
    const int64_t want = (M + p.groups - 1) / p.groups;
    return (int)(want < kPlanSms ? want : kPlanSms);
}

// Widest rows these forms take, by the backward's shared memory: 24 KB, that is 12288 columns
// of 16 bits.
constexpr int64_t kMaxRowBytes = 384 * kBwdPacks * 16;

int64_t wide_row_ranges(int64_t M, int64_t D, int vec) {
    const int64_t blocks = (D + 256 * vec - 1) / (256 * vec);
    int64_t r = (kPlanSms * 8 + blocks - 1) / blocks;
    if (r > 65535) r = 65535;
    return r < M ? r : M;
}

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }

// Bytes an element of `type` takes; 0 for an unknown type.
int type_bytes(int type) { return type == SWIGLU_FP32 ? 4 : type == SWIGLU_BF16 || type == SWIGLU_FP16 ? 2 : 0; }

bool misaligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n != 0; }

// Whether every base, row stride and the width allow 16-byte accesses.
struct Aligned {
    int size, bits = 0;
    void add(const void* p, int64_t ld) {
        if (p) bits |= (int)(reinterpret_cast<uintptr_t>(p) & 15) | (int)((ld * size) & 15);
    }
    bool ok() const { return bits == 0; }
};

// f.run<T>() for the run-time type.
template <class F>
cudaError_t with_type(int type, const F& f) {
    if (type == SWIGLU_FP32) return f.template run<float>();
    if (type == SWIGLU_FP16) return f.template run<__half>();
    return f.template run<__nv_bfloat16>();
}

template <class K>
cudaError_t allow_smem(K kern, size_t bytes) {
    return bytes <= 48 * 1024 ? cudaSuccess
                              : cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
}

struct LaunchFwd {
    const NormFwd& a;
    const NormPlan& p;
    bool shift;
    cudaStream_t s;
    template <class T, int NV, bool SHIFT, bool RES>
    cudaError_t go() const {
        // 64 (unaligned rows: 80) registers for the small CTAs, whose number hides the latencies;
        // the larger ones all hold 4 packs a thread
        auto kern = layer_norm_fwd_kernel<T, NV, SHIFT, RES, 128, SHIFT ? 6 : 8>;
        if constexpr (NV == 4) {
            if (p.threads() > 128) kern = layer_norm_fwd_kernel<T, NV, SHIFT, RES, 384, 2>;
        }
        kern<<<(unsigned)((a.M + p.groups - 1) / p.groups), p.threads(), 0, s>>>(a);
        return cudaGetLastError();
    }
    template <class T, int NV>
    cudaError_t forms() const {
        if (shift) return a.r ? go<T, NV, true, true>() : go<T, NV, true, false>();
        return a.r ? go<T, NV, false, true>() : go<T, NV, false, false>();
    }
    template <class T>
    cudaError_t run() const {
        if ((int64_t)a.D * (int)sizeof(T) > kMaxRowBytes) {
            const unsigned grid = (unsigned)(a.M < kPlanSms * 4 ? a.M : kPlanSms * 4);
            if (shift) layer_norm_fwd_wide_kernel<T, 1><<<grid, kMaxThreads, 0, s>>>(a);
            else layer_norm_fwd_wide_kernel<T, kVec<T>><<<grid, kMaxThreads, 0, s>>>(a);
            return cudaGetLastError();
        }
        return p.nv == 1 ? forms<T, 1>() : p.nv == 2 ? forms<T, 2>() : p.nv == 3 ? forms<T, 3>() : forms<T, 4>();
    }
};

struct LaunchBwd {
    const NormBwd& a;
    const NormPlan& p;
    bool shift;
    float2* sums;
    int planes;
    cudaStream_t s;
    template <class T, int NV, bool SHIFT, bool SKIP>
    cudaError_t go() const {
        auto kern = layer_norm_bwd_kernel<T, NV, SHIFT, SKIP>;
        const size_t smem = bwd_smem(p, a.D, SKIP);
        cudaError_t e = allow_smem(kern, smem);
        if (e != cudaSuccess) return e;
        kern<<<(unsigned)planes, p.threads(), smem, s>>>(a);
        return cudaGetLastError();
    }
    template <class T, int NV>
    cudaError_t forms() const {
        if (shift) return a.skip ? go<T, NV, true, true>() : go<T, NV, true, false>();
        return a.skip ? go<T, NV, false, true>() : go<T, NV, false, false>();
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
        if ((int64_t)a.D * (int)sizeof(T) > kMaxRowBytes) return shift ? wide<T, 1>() : wide<T, kVec<T>>();
        return p.nv == 1 ? forms<T, 1>() : p.nv == 2 ? forms<T, 2>() : p.nv == 3 ? forms<T, 3>() : forms<T, 4>();
    }
};

swiglu_status norm_check(int64_t M, int64_t D, int type, int param_type) {
    if (M < 0 || D <= 0) return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a size is negative or zero");
    if (M >= (int64_t(1) << 31) || D >= (int64_t(1) << 28))
        return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "layer norm: M must stay below 2^31 and D below 2^28");
    if (type_bytes(type) == 0 || (param_type != type && param_type != SWIGLU_FP32))
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: unknown type, or parameters of neither the rows' type nor fp32");
    return SWIGLU_OK;
}

}  // namespace
}  // namespace swiglu

using namespace swiglu;

extern "C" {

swiglu_status swiglu_mlp_layer_norm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr,
                                        const void* gamma, const void* beta, void* y, int64_t ldy, void* s,
                                        int64_t lds, float* mean, float* rstd, int64_t M, int64_t D, float eps,
                                        int type, int param_type, void* stream) {
    swiglu_status rc = norm_check(M, D, type, param_type);
    if (rc != SWIGLU_OK) return rc;
    if (!(eps >= 0.f)) return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: eps is negative");
    if (M == 0) return SWIGLU_OK;
    if (!x || !y) return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a required pointer is null");
    if ((residual == nullptr) != (s == nullptr) || (mean == nullptr) != (rstd == nullptr))
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: residual and s, and mean and rstd, go together");
    if (ldx < D || ldy < D || (residual && (ldr < D || lds < D)))
        return fail(SWIGLU_ERR_INVALID_ARG, "layer norm: a row stride is smaller than the width");
    const size_t n = type_bytes(type), np = type_bytes(param_type);
    if (misaligned(x, n) || misaligned(y, n) || misaligned(residual, n) || misaligned(s, n) || misaligned(gamma, np) ||
        misaligned(beta, np) || misaligned(mean, 4) || misaligned(rstd, 4))
        return fail(SWIGLU_ERR_MISALIGNED, "layer norm: a pointer is not aligned to its element");
    int sms;
    rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    Aligned v{(int)n};
    v.add(x, ldx), v.add(residual, ldr), v.add(y, ldy), v.add(s, lds), v.add(x, D);
    v.add(gamma, 0), v.add(beta, 0);
    const NormPlan p = fwd_plan(D, (int)n);
    const NormFwd a{x, residual, gamma, beta, y, s, mean, rstd, ldx, ldr, ldy, lds, M, (int)D, p.lanes,
                    param_type == SWIGLU_FP32, eps};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return launch_traced(SWIGLU_KERNEL_NORM_FWD, st, [&] { return with_type(type, LaunchFwd{a, p, !v.ok(), st}); });
}

size_t swiglu_mlp_layer_norm_bwd_workspace_size(int64_t M, int64_t D) {
    if (M <= 0 || D <= 0) return 0;
    // whatever the type and the alignment: one plane an SM, or the two-pass form's row sums and
    // the planes of its widest packs, which have the most row ranges
    const size_t narrow = 2 * round256((size_t)(M < kPlanSms ? M : kPlanSms) * D * 4);
    if (D * 4 <= kMaxRowBytes) return narrow;
    const size_t wide = round256((size_t)M * sizeof(float2)) + 2 * round256((size_t)wide_row_ranges(M, D, 8) * D * 4);
    return narrow > wide ? narrow : wide;
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
    Aligned v{(int)n};
    v.add(dy, lddy), v.add(s, lds), v.add(dskip, ldskip), v.add(dx, lddx), v.add(dy, D);
    if (D * (int64_t)n > kMaxRowBytes) v.add(gamma, 0);
    const NormPlan p = bwd_plan(M, D, (int)n, dskip != nullptr);
    const bool wide = D * (int64_t)n > kMaxRowBytes, shift = !v.ok();
    const int planes = (int)(wide ? wide_row_ranges(M, D, shift ? 1 : 16 / (int)n) : bwd_ctas(M, p));
    uint8_t* w = static_cast<uint8_t*>(workspace);
    float2* sums = reinterpret_cast<float2*>(w);
    if (wide) w += round256((size_t)M * sizeof(float2));
    float* pg = reinterpret_cast<float*>(w);
    float* pb = reinterpret_cast<float*>(w + round256((size_t)planes * D * 4));
    const NormBwd a{dy, s, gamma, dskip, mean, rstd, dx, dgamma ? pg : nullptr, dbeta ? pb : nullptr,
                    lddy, lds, ldskip, lddx, M, (int)D, p.lanes, param_type == SWIGLU_FP32};
    rc = launch_traced(SWIGLU_KERNEL_NORM_BWD, st,
                       [&] { return with_type(type, LaunchBwd{a, p, shift, sums, planes, st}); });
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
