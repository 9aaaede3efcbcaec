// moe_routed.cu -- a whole mixture-of-experts layer for a few tokens (include/swiglu_moe.h,
// swiglu_moe_routed_fwd): router, choice of experts, the chosen experts' SwiGLU blocks and
// the weighted sum per token.
//
// With at most 64 tokens the work is to read the chosen experts' weights once; the tokens
// that share an expert share that read.  Four launches, each coming up while the one before
// it ends, and nothing on the host depends on the routing: the kernels read the chosen ids and
// divide what was chosen among themselves.
//
//   route  one thread-block cluster per token: logits, softmax, top-k
//   up     per chosen expert, 8 hidden units: left and gate rows of W1 against the
//          expert's tokens, h = left * silu(gate) -> h [T * k, H] bf16 in the workspace
//   down   the steps of all chosen experts against every tile of output columns, divided
//          evenly over the CTAs; a CTA weights its part of a tile by the gates
//   join   adds the parts of every output, in a fixed order, and the residual
//
// Weights (A, 16 rows a warp) go to shared memory by asynchronous 16-byte copies and from
// there into the registers of mma.m16n8k16.  A warp copies and reads its own stages only, so
// this ring needs no barrier of the CTA.  A lane's 16 bytes hold 8 consecutive k of one row,
// and since a dot product does not care for the order of k, those 8 feed two MMAs (4 k each)
// as long as the tokens' operand B is read with the same assignment.  Copies run ahead across
// the ends of the warp's segments.  B, the rows of the tokens that chose the expert, is
// shared by the CTA: every warp reads it from a chunk in shared memory.
//
// Bound by HBM where the weights are many: 16 tokens over 8 experts of 4096 x 14336, 2 each, 2.79 GB:
// 446 us, 6.3 TB/s of the 6.78 TB/s of a copy.  Where they are few the four launches, the choice
// between them and the first and the last loads add about 20 us (one token, 8 of 64 experts of
// 2048 x 1408, 138 MB: 41 us), and where experts have many tokens each, the chunks' barriers and the
// shared memory reads of B as much again (61 tokens, 7 of 40 experts of 2056 x 1416, 698 MB: 158 us).
// One cooperative launch with barriers of the grid between the phases took as long for up to 16
// tokens and 10 us longer for 61 (a barrier of the grid costs 3 us; these launches overlap).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "convert.cuh"
#include "launch.cuh"
#include "swiglu_moe.h"

namespace swiglu {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanSms = 152;
constexpr int kMaxTokens = 64;
constexpr int kMaxTop = 16;
constexpr int kMaxExperts = 682;
constexpr int kWarps = 16, kThreads = kWarps * 32;          // one CTA an SM
constexpr int kSteps = 2;                    // steps of 64 k of a chunk
constexpr int kStages = 4;                   // steps of weights a warp has in flight or in use
constexpr int kStageBytes = 16 * 128;        // 16 rows x 64 k
constexpr int kMaxPass = 32, kMinPass = 4;   // tokens of an expert taken at a time (64 / split, at most 32)
constexpr int kEntries = kMaxExperts + kMaxTokens * kMaxTop / kMinPass;
constexpr int kRows = 64;                    // tokens x split of a chunk of B

// A chunk is STEPS * 64 k for each k group of the CTA's warps: 16 rows of weights a warp, kRows
// rows of tokens (with 64 bytes between the rows of a token).
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
__host__ __device__ constexpr int token_bytes(int steps) { return kRows * steps * 128 + kMaxPass * 64; }

struct Routed {
    const __nv_bfloat16 *x, *W1, *W2, *r;
    const void* Wr;
    __nv_bfloat16 *y, *h;
    int* ids;
    float* gates;
    int T, E, D, H, Dout, k, renorm, wr32;
    float* parts;                            // [CTA + tile][T][width]: a CTA's part of a tile
    int* span;                               // the down kernel's steps of a tile, for the join kernel
    int width, tiles, ctas;                  // output columns of a tile; tiles; CTAs of the down kernel
};



// ---------------------------------------------------------------- route

// 8 values of a row at p as fp32.
__device__ __forceinline__ void load8(float* o, const __nv_bfloat16* p) {
    load_pack<__nv_bfloat16, 8>(p).unpack(o);
}
__device__ __forceinline__ void load8(float* o, const float* p) {
    load_pack<float, 4>(p).unpack(o);
    load_pack<float, 4>(p + 4).unpack(o + 4);
}

// Order-preserving key of a logit: larger logit, larger key; NaN lowest, but above 0 (none).
__device__ __forceinline__ uint32_t logit_key(float v) {
    if (isnan(v)) return 1;
    const uint32_t u = __float_as_uint(v + 0.f);           // -0 counts as 0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Top k of a token's logits by one warp, lane's own of them in registers: lane j < k has the j-th
// choice and its gate.
template <int OWN>
__device__ __forceinline__ void choose(const Routed& a, const float* logits, int& mine, float& gate) {
    const int lane = threadIdx.x & 31;
    uint32_t key[OWN];
    float v[OWN], top = -INFINITY, sum = 0.f;
#pragma unroll
    for (int i = 0; i < OWN; ++i) {
        const bool in = lane + 32 * i < a.E;
        v[i] = in ? logits[lane + 32 * i] : -INFINITY;
        key[i] = in ? logit_key(v[i]) : 0;
        top = fmaxf(top, v[i]);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
    for (int i = 0; i < OWN; ++i)
        if (lane + 32 * i < a.E) sum += expf(v[i] - top);  // a NaN logit makes every gate NaN
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    mine = 0;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = key[0];
        int at = 0;
#pragma unroll
        for (int i = 1; i < OWN; ++i)
            if (key[i] > best) best = key[i], at = i;
        const uint32_t high = __reduce_max_sync(0xffffffffu, best);
        const int e = __reduce_min_sync(0xffffffffu, best == high ? lane + 32 * at : kMaxExperts);
#pragma unroll
        for (int i = 0; i < OWN; ++i)
            if (e == lane + 32 * i) key[i] = 0;
        if (lane == j) mine = e;
    }
    const float p = lane < a.k ? expf(logits[mine] - top) : 0.f;
    float chosen = p;
#pragma unroll
    for (int o = 16; o; o >>= 1) chosen += __shfl_xor_sync(0xffffffffu, chosen, o);
    gate = (isnan(sum) ? sum : p) / (a.renorm ? chosen : sum);
}

constexpr int kRouteWarps = 8;

// l = x Wr^T, fp32 products and sums; p = softmax(l); the top k, ties to the lowest index.  Bound by
// latencies (5.5 us alone for one token of 64 experts, of which about 2.5 are the launch).
// One cluster per token; CTA rank c computes the logits of experts c * kRouteWarps + warp,
// + cluster size * kRouteWarps, ...; the first CTA's first warp chooses.  A CTA may write another's
// shared memory only once that one is known to run: the cluster's barrier, at which all arrive first
// and wait after their first logit, which hides it.
template <class W>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(const Routed a) {
    __shared__ float logits[kMaxExperts];
    cudaTriggerProgrammaticLaunchCompletion();
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();              // this CTA runs
    const int ctas = cluster.num_blocks(), rank = cluster.block_rank();
    const int t = blockIdx.x / ctas, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* all = cluster.map_shared_rank(logits, 0);
    const __nv_bfloat16* x = a.x + (int64_t)t * a.D;
    auto logit = [&](int e) {
        const W* w = static_cast<const W*>(a.Wr) + (int64_t)e * a.D;
        float s = 0.f;
#pragma unroll 4
        for (int c = lane * 8; c < a.D; c += 256) {
            float xv[8], wv[8];
            load8(xv, x + c);
            load8(wv, w + c);
#pragma unroll
            for (int j = 0; j < 8; ++j) s += xv[j] * wv[j];
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s;
    };
    int e = rank * kRouteWarps + warp;
    float s = e < a.E ? logit(e) : 0.f;
    cluster.barrier_wait();                // every CTA runs: rank 0's shared memory may be written
    while (e < a.E) {
        if (lane == 0) all[e] = s;
        e += ctas * kRouteWarps;
        if (e < a.E) s = logit(e);
    }
    cluster.sync();
    if (rank != 0 || warp != 0) return;

    int mine;
    float gate;
    if (a.E <= 128) choose<4>(a, logits, mine, gate);
    else choose<(kMaxExperts + 31) / 32>(a, logits, mine, gate);
    if (lane < a.k) {
        a.ids[t * a.k + lane] = mine;
        a.gates[t * a.k + lane] = gate;
    }
}

// ---------------------------------------------------------------- what was chosen

// Shared by the up and the down kernel: the (token, choice) pairs sorted by expert, and within
// an expert by token, and the entries of work: up to `pass` pairs of one expert each.
struct Chosen {
    int count, most;                                       // entries; the most pairs of one
    short expert[kEntries], first[kEntries], pairs[kEntries];
    short order[kMaxTokens * kMaxTop];                     // pair = token * k + choice
};

// `scratch`: kMaxExperts x 10 bytes.  Tokens choose an expert at most once, so a bit for each
// of the 64 tokens is an expert's list, and the list's order does not depend on timing.
// The up kernel comes up while the router runs and waits for it here; only then may the down
// kernel come up, which therefore finds the router's results in place (L2) and can start on its
// weights while the last hidden units are computed.
template <bool WAIT>
__device__ __forceinline__ void read_choice(Chosen& c, const Routed& a, int pass, void* scratch) {
    unsigned long long* tokens = static_cast<unsigned long long*>(scratch);
    short* start = reinterpret_cast<short*>(tokens + kMaxExperts);
    const int pairs = a.T * a.k;
    for (int e = threadIdx.x; e < a.E; e += kThreads) tokens[e] = 0;
    if (WAIT) cudaGridDependencySynchronize();
    cudaTriggerProgrammaticLaunchCompletion();
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kThreads) atomicOr(&tokens[__ldcg(a.ids + p)], 1ull << (p / a.k));
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        int entries = 0, before = 0, most = 0;
        for (int e0 = 0; e0 < a.E; e0 += 32) {
            const int e = e0 + lane, n = e < a.E ? __popcll(tokens[e]) : 0, w = (n + pass - 1) / pass;
            int en = w, pn = n;                            // inclusive sums over the lanes
#pragma unroll
            for (int o = 1; o < 32; o *= 2) {
                const int x = __shfl_up_sync(0xffffffffu, en, o), y = __shfl_up_sync(0xffffffffu, pn, o);
                if (lane >= o) en += x, pn += y;
            }
            if (n) start[e] = (short)(before + pn - n);
            for (int i = 0; i < w; ++i) {
                const int at = entries + en - w + i, left = n - i * pass;
                c.expert[at] = (short)e;
                c.first[at] = (short)(before + pn - n + i * pass);
                c.pairs[at] = (short)min(left, pass);
            }
            most = max(most, min(n, pass));
            entries += __shfl_sync(0xffffffffu, en, 31);
            before += __shfl_sync(0xffffffffu, pn, 31);
        }
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) c.count = entries, c.most = most;
    }
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kThreads) {
        const int e = __ldcg(a.ids + p), t = p / a.k;
        c.order[start[e] + __popcll(tokens[e] & ((1ull << t) - 1))] = (short)p;
    }
    __syncthreads();
}

// ---------------------------------------------------------------- products

__device__ __forceinline__ uint4 load_smem(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void store_smem(uint32_t at, const uint4& v) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// A CTA's work is a sequence of segments: an entry's tokens against rows of its expert, over
// the steps [s, end) of 64 k.  Its kWarps warps are kWarps / split row groups x split k groups; a
// chunk is STEPS steps of each k group, that is split * STEPS * 64 consecutive k.
struct Segment {
    int entry, tile, s, end;                 // tile: the warp's 8 hidden units (up), the output tile (down)
    int first, rows;                         // of chosen.order: the pairs whose tokens are the chunk's rows
    int lead, most;                          // those before this entry's; the most pairs of one entry among them
};

// The weights of one warp, kStages steps in flight.  A copy instruction takes runs of 128 bytes
// of 4 rows (with runs of 64 bytes the launch of 16 tokens took 352 us instead of 272, with 256
// as long but fewer, larger stages 5 to 10 % longer where K is no multiple of 128).  Stage: 16
// rows of 128 bytes; odd rows have the halves exchanged, so that a quarter-warp's reads (2 rows
// x 64 bytes) touch every bank once.  `next(segment)` moves on and returns false at the end;
// `rows(segment, w, second)` gives the warp's rows 0..7 (w) and 8..15 (w + second), `ld` apart,
// and returns false where it has none.
template <int STEPS, class Next, class RowsOf>
struct Weights {
    Segment g;
    const __nv_bfloat16* w = nullptr;        // this lane's row and column 0 of a run
    int64_t second = 0, ld;
    int at = 0, half = 0, K, group, hop;     // the step copied next, and which of its chunk's it is
    bool live, mine = false;
    uint32_t copy_to, read_from, wr = 0, rd = 0;
    Next next;
    RowsOf rows;
    __device__ __forceinline__ Weights(Next n, RowsOf r, uint32_t ring, int K_, int64_t ld_, int group_, int split)
        : ld(ld_), K(K_), group(group_), hop(STEPS * split), next(n), rows(r) {
        const int lane = threadIdx.x & 31, run = lane >> 3, g8 = lane >> 2;
        ring += (threadIdx.x >> 5) * kStages * kStageBytes;
        copy_to = ring + run * 128 + (((lane & 7) * 16) ^ ((run & 1) * 64));
        read_from = ring + g8 * 128 + (((lane & 3) * 16) ^ ((g8 & 1) * 64));
        enter();
#pragma unroll
        for (int d = 0; d < kStages; ++d) issue();
    }
    __device__ __forceinline__ void enter() {
        live = next(g);
        if (!live) return;
        mine = rows(g, w, second);
        w += (int64_t)((threadIdx.x & 31) >> 3) * ld + (threadIdx.x & 7) * 8;
        at = g.s + STEPS * group;
    }
    __device__ __forceinline__ void issue() {
        if (live) {
            if (mine && at < g.end) {
                const int n = at * 64 + (int)(threadIdx.x & 7) * 8 < K ? 16 : 0;       // past the row: zeros
                const uint32_t to = copy_to + (wr & (kStages - 1)) * kStageBytes;
                const __nv_bfloat16* from = w + (n ? at * 64 : 0);
                copy(to, from, n);
                copy(to + 512, from + 4 * ld, n);
                copy(to + 1024, from + second, n);
                copy(to + 1536, from + second + 4 * ld, n);
            }
            ++at;
            if (++half == STEPS) {
                half = 0;
                at += hop - STEPS;
                if (at - STEPS * group >= g.end) enter();
            }
        }
        ++wr;
        asm volatile("cp.async.commit_group;" ::: "memory");
    }
    __device__ __forceinline__ uint32_t wait() {           // this lane's place in the step to compute
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncwarp();
        return read_from + (rd++ & (kStages - 1)) * kStageBytes;
    }
    static __device__ __forceinline__ void copy(uint32_t to, const void* from, int bytes) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
    }
};

// The tokens' rows, a chunk at a time: loaded to registers and stored to one of BUFS buffers a
// chunk ahead of that (BUFS 1: once the last chunk has been read, with a barrier more).  Buffer:
// [token][split * STEPS * 64 k], rows 64 bytes off a multiple of 128, so that the 8 rows x 64
// bytes of an MMA's operand B touch every bank once a quarter-warp.  `from(pair)`: the row of
// `base` that a pair reads.
template <int STEPS, int BUFS, class Next, class From>
struct Tokens {
    static constexpr int kPieces = kRows * STEPS * 8 / kThreads;          // 16-byte pieces a thread
    Segment g;
    const Chosen& chosen;
    const __nv_bfloat16* base;
    int at = 0, K, hop, lines, pitch;        // hop: steps of a chunk; lines: log2 of its 16-byte pieces a token
    bool live;
    uint32_t buffers, put = 0;
    uint32_t start[kPieces];                 // the first element of a piece's row in `base`; kNoRow: none
    uint4 piece[kPieces];
    Next next;
    From from;
    static constexpr uint32_t kNoRow = ~0u;  // rows x K stays below 2^31
    __device__ __forceinline__ Tokens(Next n, From f, const Chosen& c, const __nv_bfloat16* b, uint32_t smem, int K_, int split)
        : chosen(c), base(b), K(K_), buffers(smem), next(n), from(f) {
        hop = STEPS * split;
        lines = (STEPS == 2 ? 4 : 3) + (31 - __clz(split));
        pitch = (16 << lines) + 64;
        enter();
        load();
        if (BUFS == 2) {
            store();
            load();
        }
    }
    __device__ __forceinline__ void enter() {
        live = next(g);
        if (!live) return;
        at = g.s;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int i = threadIdx.x + j * kThreads, row = i >> lines;
            start[j] = row < g.rows ? (uint32_t)from(chosen.order[g.first + row]) * (uint32_t)K : kNoRow;
        }
    }
    __device__ __forceinline__ void load() {
        if (!live) return;
        const int end = g.end * 64 < K ? g.end * 64 : K, col = at * 64 + (int)(threadIdx.x & ((1 << lines) - 1)) * 8;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            piece[j] = make_uint4(0, 0, 0, 0);
            if (start[j] != kNoRow && col < end) piece[j] = *reinterpret_cast<const uint4*>(base + (start[j] + (uint32_t)col));
        }
        at += hop;
        if (at >= g.end) enter();
    }
    __device__ __forceinline__ void store() {
        const uint32_t to = buffers + (put++ & (BUFS - 1)) * token_bytes(STEPS);
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
            const int i = threadIdx.x + j * kThreads, row = i >> lines;
            if (row < kMaxPass) store_smem(to + row * pitch + (i & ((1 << lines) - 1)) * 16, piece[j]);
        }
    }
    __device__ __forceinline__ uint32_t row(const Segment& f, int i) const { return buffers + (f.lead + i) * pitch; }
};

// All rows that any pair reads, kept in the buffers' place for the whole launch where they fit:
// warps then go through their segments without a barrier a chunk.
__host__ __device__ constexpr int kept_pitch(int K) { return (K + 63) / 64 * 128 + 64; }
__host__ __device__ constexpr bool kept_fits(int64_t rows, int64_t K) {
    return rows * kept_pitch((int)K) <= 2 * token_bytes(kSteps);
}

template <class From>
struct Kept {
    const Chosen& chosen;
    uint32_t rows;
    int pitch;
    From from;
    __device__ __forceinline__ Kept(From f, const Chosen& c, const __nv_bfloat16* base, uint32_t smem, int n, int K)
        : chosen(c), rows(smem), pitch(kept_pitch(K)), from(f) {
        const int lines = (K + 63) / 64 * 8;               // 16-byte pieces of a row, the last ones zeros
        for (int i = threadIdx.x; i < n * lines; i += kThreads) {
            const int r = i / lines, c16 = i - r * lines;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (c16 * 8 < K) v = *reinterpret_cast<const uint4*>(base + (int64_t)r * K + c16 * 8);
            store_smem(rows + r * pitch + c16 * 16, v);
        }
    }
    __device__ __forceinline__ uint32_t row(const Segment& g, int i) const {
        return rows + from(chosen.order[chosen.first[g.entry] + i]) * pitch;
    }
};

// acc += this warp's part of a segment with up to NT * 8 tokens: acc[n] is rows g and g + 8 x
// tokens n * 8 + 2 q, + 1.
template <int STEPS, int BUFS, int NT, class W, class B>
__device__ __forceinline__ void products(float (*acc)[4], W& weights, B& tokens, const Segment& g, int n, bool mine,
                                         int group, int split) {
    const int lane = threadIdx.x & 31;
    uint32_t row[NT];                        // of token n * 8 + g in a buffer; past the last, the last's
#pragma unroll
    for (int i = 0; i < NT; ++i)
        row[i] = tokens.row(g, min(i * 8 + (lane >> 2), n - 1)) + group * STEPS * 128 + (lane & 3) * 16;
    for (int c = g.s; c < g.end; c += STEPS * split) {
        uint32_t buffer = c * 128;           // kept rows: the chunk's place in them
        if constexpr (BUFS > 0) {
            __syncthreads();                 // the last chunk's tokens are read, and (BUFS 2) this chunk's stored
            buffer = BUFS == 1 ? 0 : (tokens.put & 1 ? 0 : 1) * token_bytes(STEPS);        // stored last
            tokens.store();
            if (BUFS == 1) __syncthreads();
            tokens.load();
        }
#pragma unroll
        for (int d = 0; d < STEPS; ++d) {
            const uint32_t from = weights.wait();
            if (mine && c + STEPS * group + d < g.end) {
                const uint4 w0 = load_smem(from), w1 = load_smem(from + 1024), w2 = load_smem(from ^ 64), w3 = load_smem((from + 1024) ^ 64);
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const uint4 u = load_smem(row[i] + buffer + d * 128), v = load_smem(row[i] + buffer + d * 128 + 64);
                    mma(acc[i], w0.x, w1.x, w0.y, w1.y, u.x, u.y);
                    mma(acc[i], w0.z, w1.z, w0.w, w1.w, u.z, u.w);
                    mma(acc[i], w2.x, w3.x, w2.y, w3.y, v.x, v.y);
                    mma(acc[i], w2.z, w3.z, w2.w, w3.w, v.z, v.w);
                }
            }
            __syncwarp();                    // every lane has read the stage that is filled next
            weights.issue();
        }
    }
}

// products() over the number of 8-token tiles that the most tokens of one of the chunk's entries
// take (the same for all warps, which meet at its barriers).  An expert of 17 to 24 tokens takes
// three tiles: with two and four only, 61 ragged tokens took 164 us instead of 158.
template <int STEPS, int BUFS, class W, class B>
__device__ __forceinline__ void products_of(float (*acc)[4], W& weights, B& tokens, const Segment& g, int n, bool mine,
                                            int group, int split) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    if (g.most <= 8) products<STEPS, BUFS, 1>(acc, weights, tokens, g, n, mine, group, split);
    else if (g.most <= 16) products<STEPS, BUFS, 2>(acc, weights, tokens, g, n, mine, group, split);
    else if (g.most <= 24) products<STEPS, BUFS, 3>(acc, weights, tokens, g, n, mine, group, split);
    else products<STEPS, BUFS, 4>(acc, weights, tokens, g, n, mine, group, split);
}

// h = left * silu(gate), [left | gate] = x W1^T of the expert.  Bound by HBM: 16 tokens, 8 experts of
// 4096 x 14336, 1.88 GB in 288 us, 6.5 TB/s.
// A segment is, for a warp, 8 hidden units (`tile`) of an entry's expert over the whole of D:
// MMA rows 0..7 are their left rows of W1, rows 8..15 the gate rows of the same units, so a
// lane ends with left and gate of its unit.  KEPT: the tokens stay in shared memory, and the
// units of all entries are dealt to the warps one by one; otherwise a CTA's row groups take
// neighbouring units of one entry, which share its chunks of tokens.
constexpr int kUpSmem = kRingBytes + 2 * token_bytes(kSteps) + kWarps * 16 * 32 * 4;

template <bool KEPT>
__global__ void __launch_bounds__(kThreads, 1) moe_up_kernel(const Routed a) {
    __shared__ Chosen chosen;
    extern __shared__ __align__(128) unsigned char smem[];
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem);
    auto from = [&](int pair) { return pair / a.k; };
    // x is older than the launch ahead of this one
    Kept<decltype(from)> kept(from, chosen, a.x, ring + kRingBytes, KEPT ? a.T : 0, a.D);
    read_choice<true>(chosen, a, kMaxPass, smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int groups = a.H / 8, units = chosen.count * groups, steps = (a.D + 63) / 64, ctas = gridDim.x;
    int split = 1;
    float least = INFINITY;
    for (int s = 1; s <= kWarps && (KEPT || s * chosen.most <= kRows); s *= 2) {
        if (KEPT) {
            // In units of a warp's time for a unit of 32 D bytes, at the 6.8 KB/us its copies in flight
            // bring: all full rounds at the HBM rate, the last, partial one at that or at a warp's
            // (4 tokens, 30 of 64 experts of 2048 x 1408: split 1 99.5 us, 2 94.6; one token, 8 of
            // them: 41.8, 47.0), and 0.5 us a round for adding the k groups' sums.  (With the
            // compiler's exact divisions, finding this out took 1.2 us.)
            const float warps = (float)(ctas * kWarps), hbm = 1.015e-3f * (float)units, inv = __fdividef(1.f, (float)s);
            const float rounds = __fdividef((float)units * (float)s, warps), full = floorf(rounds);
            // hbm / rounds: a round of all warps at the HBM rate
            const float each = 1.015e-3f * warps * inv, part = rounds - full;
            const float cost = each * full + (part > 0.f ? fmaxf(inv, each * part) : 0.f) +
                               (s > 1 ? __fdividef(106.f * (full + 1.f), (float)a.D) : 0.f);
            if (cost < least) least = cost, split = s;
            if (rounds <= 1.f && hbm * (float)s >= 1.f) break;             // one round, at the HBM rate
        } else {
            // the split whose last round of a CTA's units wastes least (a segment's end costs
            // about a chunk), among those whose chunk of tokens fits
            const float mine = __fdividef((float)units * (float)s, (float)(ctas * kWarps));
            const float cost = ceilf(mine) * (__fdividef(1.f, (float)s) + __fdividef(2.f, (float)steps));
            if (cost < least) least = cost, split = s;
        }
    }
    const int per = kWarps / split, row = warp / split, group = warp % split;
    // KEPT: round j of a warp is unit (j * per + row) * ctas + CTA.  Otherwise a CTA has an even,
    // consecutive share of the units and takes `per` at a time, of more than one entry where their
    // tokens, which follow one another in the list, fit a chunk together (cut at every entry's end,
    // the CTAs with such an end took a round more: 61 ragged tokens 171 us instead of 165).
    const int begin = KEPT ? 0 : (int)((int64_t)units * blockIdx.x / ctas);
    const int end = KEPT ? (units + ctas * per - 1) / (ctas * per) : (int)((int64_t)units * (blockIdx.x + 1) / ctas);
    auto segment = [&](int& at, Segment& f) {
        if (at >= end) return false;
        if (KEPT) {
            const int u = (at++ * per + row) * ctas + blockIdx.x, entry = u / groups;
            f = {entry, u < units ? u % groups : groups, 0, steps, 0, 0, 0, u < units ? chosen.pairs[entry] : 0};
            return true;
        }
        const int entry0 = at / groups, u = at + row;
        int n = min(per, end - at), rows = 0, most = 0, entry = entry0, lead = 0;
        for (int e = entry0, next = (entry0 + 1) * groups;; ++e, next += groups) {
            const int pairs = chosen.pairs[e];
            if (e > entry0 && rows + pairs > min(kMaxPass, kRows / split)) {
                n = min(n, next - groups - at);            // its units are another chunk's
                break;
            }
            if (u >= next - groups) entry = e, lead = rows;
            rows += pairs;
            most = max(most, pairs);
            if (next >= at + n) break;
        }
        f = {entry, row < n ? u - entry * groups : groups, 0, steps, chosen.first[entry0], rows, lead, most};
        at += n;
        return true;
    };
    int ahead_w = begin, ahead_t = begin;
    auto next_w = [&](Segment& f) { return segment(ahead_w, f); };
    auto next_t = [&](Segment& f) { return segment(ahead_t, f); };
    auto rows = [&](const Segment& f, const __nv_bfloat16*& w, int64_t& second) {
        if (f.tile >= groups) return false;  // this warp has no unit in the segment
        w = a.W1 + ((int64_t)chosen.expert[f.entry] * 2 * a.H + f.tile * 8) * a.D;
        second = (int64_t)a.H * a.D;
        return true;
    };
    float* part = reinterpret_cast<float*>(smem + kRingBytes + 2 * token_bytes(kSteps));       // [warp][value][lane]
    Weights<kSteps, decltype(next_w), decltype(rows)> weights(next_w, rows, ring, a.D, a.D, group, split);
    auto run = [&](auto& tokens, auto bufs) {
        int at = begin;
        for (Segment f; segment(at, f);) {
            const bool mine = f.tile < groups;
            if (KEPT && !mine && split == 1) break;
            const int n = KEPT && !mine ? 0 : chosen.pairs[f.entry], unit = f.tile * 8 + g;
            float acc[4][4];
            if (!KEPT || mine) products_of<kSteps, decltype(bufs)::value>(acc, weights, tokens, f, n, mine, group, split);
            if (split > 1) {
                if (group > 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i * 8 < n)
#pragma unroll
                            for (int v = 0; v < 4; ++v) part[(warp * 16 + i * 4 + v) * 32 + lane] = acc[i][v];
                }
                __syncthreads();             // (unless KEPT, the next segment's first chunk has one before part is written again)
                if (group == 0) {
                    for (int p = 1; p < split; ++p)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (i * 8 < n)
#pragma unroll
                                for (int v = 0; v < 4; ++v) acc[i][v] += part[((warp + p) * 16 + i * 4 + v) * 32 + lane];
                }
                if (KEPT) __syncthreads();
            }
            if (mine && group == 0) {
                // h is rounded to bf16 once, for the down product's MMA, as the block's forward does (y is then
                // off by up to 0.0024 of its norm, by 0.0017 with h in 32 bits); left and gate stay fp32.
                // __expf is off by less than 2^-16 of its value, far below that rounding.
#pragma unroll
                for (int i = 0; i < 4; ++i) {
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const int col = i * 8 + 2 * q + v;
                        if (col < n) {
                            const float left = acc[i][v], gate = acc[i][2 + v];
                            a.h[(int64_t)chosen.order[chosen.first[f.entry] + col] * a.H + unit] =
                                __float2bfloat16_rn(left * (gate / (1.f + __expf(-gate))));
                        }
                    }
                }
            }
        }
    };
    if constexpr (KEPT) {
        run(kept, std::integral_constant<int, 0>{});       // read_choice's barriers have published the rows
    } else {
        Tokens<kSteps, 2, decltype(next_t), decltype(from)> tokens(next_t, from, chosen, a.x, ring + kRingBytes, a.D, split);
        run(tokens, std::integral_constant<int, 2>{});
    }
}

// CTAs of the down kernel that have steps: CTA c has [all * c / n, all * (c + 1) / n) of all =
// tiles * span steps, at least one each.
__device__ __forceinline__ int down_sharers(int ctas, int tiles, int span) {
    return (int)min((long long)ctas, (long long)tiles * span);
}

// Parts of y = sum gate * (h W2^T).  Bound by HBM: as above 0.94 GB in 150 us, 6.3 TB/s.
// A tile is `width` = 16 * (kWarps / split) output columns, and its span the steps of all
// entries, one after the other; the spans of all tiles are divided evenly over the CTAs.  A
// warp adds each segment's sums, times the gates, into its own fp32 tile [T][16]; at the end
// of a tile (or of the CTA's steps) the warps' are added in order and stored as a part.
// (Clusters whose CTAs shared a tile and added in distributed shared memory were tried: at
// most 128 of the 152 SMs fit whole clusters, and 61 ragged tokens took 86 us instead of 70.)
// BUFS 0: the hidden rows are kept in shared memory.
template <int BUFS>
__global__ void __launch_bounds__(kThreads, 1) moe_down_kernel(const Routed a, int split) {
    __shared__ Chosen chosen;
    extern __shared__ __align__(128) unsigned char smem[];
    read_choice<false>(chosen, a, min(kMaxPass, kRows / split), smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
    const int steps = (a.H + 63) / 64, row = warp / split, group = warp % split;
    const int span = chosen.count * steps, sharers = down_sharers(a.ctas, a.tiles, span);
    const long long all = (long long)a.tiles * span;
    const long long begin = (int)blockIdx.x < sharers ? all * blockIdx.x / sharers : 0;
    const long long end = (int)blockIdx.x < sharers ? all * (blockIdx.x + 1) / sharers : 0;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.span = span;
    struct Cursor {
        int left, tile, entry, step;         // steps left to the CTA; the next one
    };
    const int tile0 = (int)(begin / span), in0 = (int)(begin - (long long)tile0 * span), entry0 = in0 / steps;
    const Cursor start{(int)(end - begin), tile0, entry0, in0 - entry0 * steps};
    Cursor ahead_w = start, ahead_t = start;
    auto segment = [&](Cursor& c, Segment& f) {
        if (c.left == 0) return false;
        const int n = min(steps - c.step, c.left);
        f = {c.entry, c.tile, c.step, c.step + n, chosen.first[c.entry], chosen.pairs[c.entry], 0, chosen.pairs[c.entry]};
        c.left -= n;
        c.step += n;
        if (c.step == steps) {
            c.step = 0;
            if (++c.entry == chosen.count) c.entry = 0, ++c.tile;
        }
        return true;
    };
    auto next_w = [&](Segment& f) { return segment(ahead_w, f); };
    auto next_t = [&](Segment& f) { return segment(ahead_t, f); };
    auto rows = [&](const Segment& f, const __nv_bfloat16*& w, int64_t& second) {
        const int out = f.tile * a.width + row * 16;
        if (out >= a.Dout) return false;
        w = a.W2 + ((int64_t)chosen.expert[f.entry] * a.Dout + out) * a.H;
        second = out + 8 < a.Dout ? 8 * (int64_t)a.H : 0;              // Dout is a multiple of 8
        return true;
    };
    auto from = [&](int pair) { return pair; };
    const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem);
    float* sums = reinterpret_cast<float*>(smem + kRingBytes + (BUFS == 1 ? 1 : 2) * token_bytes(kSteps));      // [kWarps][T][16]
    float* tile = sums + warp * a.T * 16;
    Weights<kSteps, decltype(next_w), decltype(rows)> weights(next_w, rows, ring, a.H, a.H, group, split);
    for (int i = lane; i < a.T * 16; i += 32) tile[i] = 0.f;
    cudaGridDependencySynchronize();         // h is complete; the first weights are on their way
    auto finish = [&](int t) {               // tile t's part, and zeros for the next
        __syncthreads();
        float* part = a.parts + (int64_t)(blockIdx.x + t) * a.T * a.width;
        for (int i = threadIdx.x; i < a.T * a.width; i += kThreads) {
            const int c = i % a.width;
            float* p = sums + c / 16 * split * a.T * 16 + i / a.width * 16 + c % 16;
            float v = 0.f;
            for (int w = 0; w < split; ++w) {
                v += p[w * a.T * 16];
                p[w * a.T * 16] = 0.f;
            }
            part[i] = v;
        }
        __syncthreads();
    };
    auto run = [&](auto& tokens) {
        Cursor at = start;
        int open = -1;
        for (Segment f; segment(at, f);) {
            if (open >= 0 && f.tile != open) finish(open);
            open = f.tile;
            const int n = chosen.pairs[f.entry], first = chosen.first[f.entry];
            const bool mine = f.tile * a.width + row * 16 < a.Dout;
            float acc[4][4];
            products_of<kSteps, BUFS>(acc, weights, tokens, f, n, mine, group, split);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const int col = i * 8 + 2 * q + v;
                    if (col < n) {
                        const int p = chosen.order[first + col];
                        const float gate = __ldcg(a.gates + p);
                        float* o = tile + p / a.k * 16 + g;
                        o[0] += gate * acc[i][v];
                        o[8] += gate * acc[i][2 + v];
                    }
                }
            }
            __syncwarp();
        }
        if (open >= 0) finish(open);
    };
    if constexpr (BUFS == 0) {
        Kept<decltype(from)> kept(from, chosen, a.h, ring + kRingBytes, a.T * a.k, a.H);
        __syncthreads();
        run(kept);
    } else {
        Tokens<kSteps, BUFS, decltype(next_t), decltype(from)> tokens(next_t, from, chosen, a.h, ring + kRingBytes, a.H, split);
        run(tokens);
    }
}

// Bound by latency: about 2 us beside its launch.  y: the parts of a tile, in the order of the CTAs whose steps meet its span, that is
// first <= c <= last with first = floor((tile * span * n + n - 1) / (tiles * span)) and
// last = ceil((tile + 1) * n / tiles) - 1.  Grid (blocks of columns, tokens).
__global__ void __launch_bounds__(256) moe_join_kernel(const Routed a) {
    const int col = blockIdx.x * 256 + threadIdx.x, tile = col / a.width, in = col - tile * a.width;
    const int64_t i = (int64_t)blockIdx.y * a.Dout + col;
    const float* part = a.parts + (int64_t)blockIdx.y * a.width + in;
    const float v = a.r && col < a.Dout ? to_f32(a.r[i]) : 0.f;            // older than the call
    cudaGridDependencySynchronize();
    if (col >= a.Dout) return;
    const int span = *a.span, n = down_sharers(a.ctas, a.tiles, span);
    const int first = (tile * n + (n - 1) / span) / a.tiles, last = ((tile + 1) * n - 1) / a.tiles;
    float sum = 0.f;
    for (int c = first; c <= last; c += 8) {               // 8 loads in flight
        float p[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = c + j <= last ? part[(int64_t)(c + j + tile) * a.T * a.width] : 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum += p[j];
    }
    a.y[i] = __float2bfloat16_rn(v + sum);
}

// ---------------------------------------------------------------- host side

bool width_ok(int64_t v) { return v > 0 && v % 8 == 0 && v < (int64_t(1) << 24); }

// A grid of clusters of `size` CTAs along x; early: the launch may start before the one ahead of it ends.
template <class... Args>
cudaError_t launch_clusters(void (*kernel)(Args...), dim3 clusters, int size, int threads, size_t smem, cudaStream_t s,
                            bool early, Args... args) {
    const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = size;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 2 : 1;
    cfg.gridDim = dim3(clusters.x * size, clusters.y);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int down_smem(int bufs, int64_t T) {
    return kRingBytes + bufs * token_bytes(kSteps) + (int)(kWarps * T * 16 * sizeof(float));
}

// Output columns of a tile: as many as leave 12 tiles (wide tiles share the tokens' chunks among
// more warps; few tiles have many parts each to add).
int down_width(int64_t Dout) {
    int width = kWarps * 16;
    while (width > 16 && (Dout + width - 1) / width < 12) width /= 2;
    return width;
}
int down_tiles(int64_t Dout) { return (int)((Dout + down_width(Dout) - 1) / down_width(Dout)); }
int down_ctas(int64_t Dout) { return std::min(kPlanSms, 16 * down_tiles(Dout)); }

size_t round256(size_t v) { return (v + 255) & ~size_t(255); }
constexpr size_t kSpanBytes = 256;           // the join kernel's span
size_t h_bytes(int64_t T, int64_t H, int64_t k) { return round256((size_t)T * (size_t)k * (size_t)H * 2); }
size_t part_bytes(int64_t T, int64_t Dout) {
    return (size_t)(down_ctas(Dout) + down_tiles(Dout)) * (size_t)T * (size_t)down_width(Dout) * sizeof(float);
}

}  // namespace
}  // namespace swiglu

using namespace swiglu;

extern "C" {

size_t swiglu_moe_routed_fwd_workspace_size(int64_t T, int64_t H, int64_t Dout, int64_t top_k) {
    if (T <= 0 || H <= 0 || Dout <= 0 || top_k <= 0) return 0;
    return h_bytes(T, H, top_k) + kSpanBytes + round256(part_bytes(T, Dout));
}

swiglu_status swiglu_moe_routed_fwd(const void* x, const void* Wr, const void* W1, const void* W2,
                                    const void* residual, void* y, int32_t* ids, float* gates, int64_t T, int64_t E,
                                    int64_t D, int64_t H, int64_t Dout, int64_t top_k, int renormalize,
                                    int router_fp32, void* workspace, size_t workspace_bytes, void* stream) {
    if (T < 0 || E <= 0 || D <= 0 || H <= 0 || Dout <= 0 || top_k <= 0 || top_k > E)
        return fail(SWIGLU_ERR_INVALID_ARG, "routed layer: a size is negative or zero, or top_k above E");
    if (T > kMaxTokens || E > kMaxExperts || top_k > kMaxTop || !width_ok(D) || !width_ok(H) || !width_ok(Dout))
        return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "routed layer: needs T <= 64, E <= 682, top_k <= 16 and widths that are multiples of 8 below 2^24");
    if (T == 0) return SWIGLU_OK;
    if (T * top_k * H >= (int64_t(1) << 31)) return fail(SWIGLU_ERR_UNSUPPORTED_SHAPE, "routed layer: T * top_k * H must stay below 2^31");
    if (!x || !Wr || !W1 || !W2 || !y || !ids || !gates || !workspace)
        return fail(SWIGLU_ERR_INVALID_ARG, "routed layer: a required pointer is null");
    if (!aligned16(x) || !aligned16(Wr) || !aligned16(W1) || !aligned16(W2) || !aligned16(residual) || !aligned16(y) ||
        !aligned16(workspace) || (reinterpret_cast<uintptr_t>(ids) & 3) || (reinterpret_cast<uintptr_t>(gates) & 3))
        return fail(SWIGLU_ERR_MISALIGNED, "routed layer: a pointer is not 16-byte aligned (ids, gates: 4)");
    if (workspace_bytes < swiglu_moe_routed_fwd_workspace_size(T, H, Dout, top_k))
        return fail(SWIGLU_ERR_WORKSPACE_TOO_SMALL, "routed layer: workspace smaller than the size query returns");
    int sms;
    swiglu_status rc = device_sms(&sms);
    if (rc != SWIGLU_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    typedef const __nv_bfloat16* In;
    uint8_t* ws = static_cast<uint8_t*>(workspace) + h_bytes(T, H, top_k);
    const Routed a{(In)x, (In)W1, (In)W2, (In)residual, Wr, (__nv_bfloat16*)y, (__nv_bfloat16*)workspace, ids, gates,
                   (int)T, (int)E, (int)D, (int)H, (int)Dout, (int)top_k, renormalize != 0, router_fp32 != 0,
                   reinterpret_cast<float*>(ws + kSpanBytes), reinterpret_cast<int*>(ws), down_width(Dout), down_tiles(Dout),
                   down_ctas(Dout)};
    // route: up to 8 CTAs of 8 warps share a token's experts
    const int route_ctas = E <= 8 ? 1 : E <= 16 ? 2 : E <= 32 ? 4 : 8;
    rc = launch_traced(SWIGLU_KERNEL_MOE_ROUTE, s, [&] {
        return launch_clusters(router_fp32 ? moe_route_kernel<float> : moe_route_kernel<__nv_bfloat16>, (int)T, route_ctas,
                               kRouteWarps * 32, 0, s, false, a);
    });
    if (rc != SWIGLU_OK) return rc;
    rc = launch_traced(SWIGLU_KERNEL_MOE_UP, s, [&] {
        return kept_fits(T, D) ? launch_clusters(moe_up_kernel<true>, kPlanSms, 1, kThreads, kUpSmem, s, true, a)
                               : launch_clusters(moe_up_kernel<false>, kPlanSms, 1, kThreads, kUpSmem, s, true, a);
    });
    if (rc != SWIGLU_OK) return rc;
    rc = launch_traced(SWIGLU_KERNEL_MOE_DOWN, s, [&] {
        const int split = kWarps * 16 / a.width;
        if (T <= 32 && kept_fits(T * top_k, H))
            return launch_clusters(moe_down_kernel<0>, a.ctas, 1, kThreads, down_smem(2, T), s, true, a, split);
        // two buffers of tokens where their sums leave room
        return T <= 32 ? launch_clusters(moe_down_kernel<2>, a.ctas, 1, kThreads, down_smem(2, T), s, true, a, split)
                       : launch_clusters(moe_down_kernel<1>, a.ctas, 1, kThreads, down_smem(1, T), s, true, a, split);
    });
    if (rc != SWIGLU_OK) return rc;
    return launch_traced(SWIGLU_KERNEL_MOE_JOIN, s, [&] {
        return launch_clusters(moe_join_kernel, dim3((unsigned)((Dout + 255) / 256), (unsigned)T), 1, 256, 0, s, true, a);
    });
}

}  // extern "C"
