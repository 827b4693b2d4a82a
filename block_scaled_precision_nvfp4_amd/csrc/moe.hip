// moe.hip -- the way of tokens to their experts and back.  A token has k slots, slot i = t k + j being its
// j-th expert's:
//
//   sort      c_g slots want expert g; group g starts at a multiple of `align`, and a slot's row is its group's start
//             plus the slots before it that want the same expert (a stable counting sort)
//   gather    out[row of slot i] = x[i / k], as bf16, row-scaled NVFP4 or MXFP8; rows of no slot are zero
//   combine   out[t] = sum_j w[t][j] y[row of slot t k + j]
//   backward  dy[row of slot i] = w_i dout[i / k],  dw_i = <dout[i / k], y[row of slot i]>
//
// None of them does arithmetic to speak of: a call is bound by the bytes of its rows, or by latency.  us in a graph, with
// several inputs in turn (the caches hold one): sort 37 x 2 slots of 8 experts 3.8, 16384 x 8 of 128 11.0 (two
// launches); gather 16384 x 2 of 4096 bf16 70 (5.8 TB/s), 8191 x 8 of 2080 MXFP8 34 (5.2), 64 x 8 of 4096 NVFP4 3.4;
// combination 1 x 2 of 4096 2.2, 16384 x 2 63 (6.4); its backward 16384 x 2 121 (5.6), 333 x 6 of 1032 fp32 6.1.  A
// large copy runs at 4.8 to 4.9.
#include "encode.hpp"
#include "launch.hpp"

namespace bsq {

// ---------------------------------------------------------------- sort

constexpr int SORT_WAVES = 16;
constexpr int SORT_HIST = 8192;        // counters of a workgroup: its waves' times the experts
constexpr int SORT_KEEP = 16;          // slots of a lane that stay in registers

struct SortArgs {
    const void* experts;   // ids of 4 or 8 bytes
    int id8;
    int64_t n;
    int E;
    int align;             // a power of two
    int64_t rows;
    int64_t* offsets;
    int32_t* positions;
    int32_t* source;
    int32_t* counts;       // [workgroups][E], with several workgroups
    int64_t mine;          // slots of a wave, one after another, a multiple of 64
};

// A slot's expert, E for one that is dropped.
__device__ __forceinline__ int sort_id(const SortArgs& a, int64_t i) {
    const int64_t id = a.id8 ? ((const int64_t*)a.experts)[i] : (int64_t)((const int32_t*)a.experts)[i];
    return id >= 0 && id < a.E ? (int)id : a.E;
}

// The lanes of the wave whose id (of `bits` bits) is this lane's.
__device__ __forceinline__ uint64_t same_id(int id, int bits) {
    uint64_t m = ~0ull;
    for (int b = 0; b < bits; ++b) {
        const uint64_t one = __ballot((id >> b) & 1);
        m &= ((id >> b) & 1) ? one : ~one;
    }
    return m;
}

// A slot's rank among its expert's slots of the wave so far, which next[id] counts; one lane of each expert counts
// for all (an atomic, of the wave's own counter, only so that it also returns the count before).
__device__ __forceinline__ int take_rank(int* next, int id, int E, int bits, int lane) {
    const uint64_t m = same_id(id, bits);
    const int leader = __builtin_ctzll(m);
    int at = 0;
    if (id < E && lane == leader) at = atomicAdd(&next[id], __popcll(m));
    return __shfl(at, leader) + __popcll(m & ((1ull << lane) - 1));
}

__global__ __launch_bounds__(64 * SORT_WAVES) void moe_count_kernel(SortArgs a) {
    __shared__ int hist[1024];
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) hist[e] = 0;
    __syncthreads();
    const int bits = 32 - __builtin_clz(a.E);
    const int64_t chunk = a.mine * (blockDim.x >> 6), first = (int64_t)blockIdx.x * chunk;
    for (int64_t c = 0; c < chunk; c += blockDim.x) {
        const int64_t i = first + c + threadIdx.x;
        const int id = i < a.n ? sort_id(a, i) : a.E;
        const uint64_t m = same_id(id, bits);
        if (id < a.E && (int)(threadIdx.x & 63) == __builtin_ctzll(m)) atomicAdd(&hist[id], __popcll(m));
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += blockDim.x) a.counts[(int64_t)blockIdx.x * a.E + e] = hist[e];
}

// A workgroup places its waves' slots: their ranks within the wave, the slots before the wave (from the other
// workgroups' counts and the workgroup's own), and the groups' starts.  KEEP: at most SORT_KEEP slots a lane, whose
// experts and ranks stay in registers in between; otherwise they are read and counted again.
template <bool KEEP>
__global__ __launch_bounds__(64 * SORT_WAVES) void moe_place_kernel(SortArgs a) {
    __shared__ int next[SORT_HIST];                    // [wave][E]: the wave's count, then its next row, of each expert
    __shared__ int start[1024], total[1024], before[1024];
    __shared__ int sums[SORT_WAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6, E = a.E;
    const int bits = 32 - __builtin_clz(E);
    const int64_t first = ((int64_t)blockIdx.x * waves + wave) * a.mine;
    int id[SORT_KEEP], rank[SORT_KEEP];
    if constexpr (KEEP) {
#pragma unroll
        for (int u = 0; u < SORT_KEEP; ++u) {
            const int64_t i = first + 64 * u + lane;
            id[u] = 64 * u < a.mine && i < a.n ? sort_id(a, i) : E;
        }
    }
    for (int i = threadIdx.x; i < waves * E; i += blockDim.x) next[i] = 0;
    for (int e = threadIdx.x; e < E; e += blockDim.x) total[e] = before[e] = 0;
    __syncthreads();
    if (gridDim.x > 1) {   // an expert's counts dealt to as many threads as there are
        const int group = 1 << (E > 1 ? 32 - __builtin_clz(E - 1) : 0);   // E <= 1024
        const int parts = blockDim.x / group > 0 ? blockDim.x / group : 1;
        for (int e = threadIdx.x % group; e < E; e += blockDim.x) {   // more than one round with parts == 1 only
            int s = 0, b = 0;
            const int p = parts > 1 ? threadIdx.x / group : 0;
#pragma unroll 8
            for (int g = p; g < (int)gridDim.x; g += parts) {
                const int v = a.counts[(int64_t)g * E + e];
                s += v;
                b += g < (int)blockIdx.x ? v : 0;
            }
            atomicAdd(&total[e], s);
            atomicAdd(&before[e], b);
        }
    }
    if constexpr (KEEP) {
#pragma unroll
        for (int u = 0; u < SORT_KEEP; ++u)
            if (64 * u < a.mine) rank[u] = take_rank(next + wave * E, id[u], E, bits, lane);
    } else {
        for (int64_t c = 0; c < a.mine; c += 64) {
            const int64_t i = first + c + lane;
            take_rank(next + wave * E, i < a.n ? sort_id(a, i) : E, E, bits, lane);
        }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += blockDim.x) {   // what a wave starts from; the group's start comes on top
        int at = before[e];
        for (int w = 0; w < waves; ++w) {
            const int c = next[w * E + e];
            next[w * E + e] = at;
            at += c;
        }
        if (gridDim.x == 1) total[e] = at;
    }
    __syncthreads();
    // the groups' starts: a running sum of the padded totals, a stretch of experts after another
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += blockDim.x) {
        const int e = e0 + threadIdx.x;
        const int padded = e < E ? (total[e] + a.align - 1) & -a.align : 0;
        int v = padded;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            const int u = __shfl_up(v, o);
            if (lane >= o) v += u;
        }
        if (lane == 63) sums[wave] = v;
        __syncthreads();
        int at = base, all = 0;
        for (int w = 0; w < waves; ++w) {
            if (w < wave) at += sums[w];
            all += sums[w];
        }
        if (e < E) start[e] = at + v - padded;
        base += all;
        __syncthreads();
    }
    if (blockIdx.x == 0) {
        for (int e = threadIdx.x; e < E; e += blockDim.x) a.offsets[e] = start[e];
        if (threadIdx.x == 0) a.offsets[E] = base;
    }
    auto place = [&](int64_t i, int e, int at) {
        if (i >= a.n) return;
        a.positions[i] = e < E ? at : -1;
        if (e < E) a.source[at] = (int32_t)i;
    };
    if constexpr (KEEP) {
#pragma unroll
        for (int u = 0; u < SORT_KEEP; ++u)
            if (64 * u < a.mine)
                place(first + 64 * u + lane, id[u], id[u] < E ? start[id[u]] + next[wave * E + id[u]] + rank[u] : 0);
    } else {
        for (int64_t c = 0; c < a.mine; c += 64) {
            const int64_t i = first + c + lane;
            const int e = i < a.n ? sort_id(a, i) : E;
            const int at = take_rank(next + wave * E, e, E, bits, lane);
            place(i, e, e < E ? start[e] + at : 0);
        }
    }
    // rows of no slot: the groups' padding, and what lies behind the last group
    const int shift = __builtin_ctz(a.align);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < (int64_t)E << shift; i += (int64_t)gridDim.x * blockDim.x) {
        const int e = (int)(i >> shift), r = start[e] + total[e] + (int)(i & (a.align - 1));
        if (r < (e + 1 < E ? start[e + 1] : base)) a.source[r] = -1;
    }
    for (int64_t r = base + (int64_t)blockIdx.x * blockDim.x + threadIdx.x; r < a.rows; r += (int64_t)gridDim.x * blockDim.x)
        a.source[r] = -1;
}

// The launch's shape: one workgroup up to 4096 slots, of as many waves as have slots; else a count first, and
// several workgroups, each wave with 64 slots or, where that would be over 128 workgroups, more.  us in a graph, one
// workgroup and several, 8 / 128 experts: 2048 slots 6.1 / 7.7 and 8.2 / 9.3, 4096 7.5 / 9.8 and 8.2 / 9.1 (a
// second launch costs the host 2), 16384 16.2 / 22.1 and 8.4 / 9.6; with 128 slots a wave 9.5 / 11.1.  Of 256 / 1000
// experts 2048 slots take 8.5 / 16.2 and 9.7 / 12.8, 4096 10.8 / 19.7 and 9.6 / 11.1: there several workgroups would pay
// earlier, and the limit does not look at the experts.  A few slots of
// many experts take a wave for 16 experts too, which share their counts: 4 x 5 of 63, padded to 32, 7.0 and 5.1.
constexpr int SORT_ONE = 4096, SORT_MINE = 64;

struct SortShape {
    int64_t groups, mine;
    int waves;
};

static SortShape sort_shape(int64_t n, int64_t E) {
    int waves = SORT_WAVES;
    while (waves * E > SORT_HIST) waves /= 2;
    if (n <= SORT_ONE) {
        while (waves > 1 && waves / 2 * 64 >= n && waves / 2 * 16 >= E) waves /= 2;
        const int64_t lanes = 64 * waves;
        return {1, (n + lanes - 1) / lanes * 64, waves};
    }
    int64_t mine = SORT_MINE;
    while ((n + mine * waves - 1) / (mine * waves) > 128) mine *= 2;
    return {(n + mine * waves - 1) / (mine * waves), mine, waves};
}

int64_t moe_sort_counts(int64_t n, int64_t E) {
    const int64_t groups = sort_shape(n, E).groups;
    return groups > 1 ? groups * E : 0;
}

int launch_moe_sort(const void* experts, int id8, int64_t n, int64_t E, int64_t align, int64_t rows, int64_t* offsets,
                    int32_t* positions, int32_t* source, int32_t* counts, void* hip_stream) {
    hipStream_t s = (hipStream_t)hip_stream;
    const SortShape h = sort_shape(n, E);
    const SortArgs a{experts, id8, n, (int)E, (int)align, rows, offsets, positions, source, counts, h.mine};
    const dim3 grid((unsigned)h.groups), block(64 * h.waves);
    if (h.groups > 1) {
        hipLaunchKernelGGL(moe_count_kernel, grid, block, 0, s, a);
        const int e = (int)hipGetLastError();
        if (e) return e;
    }
    if (h.mine <= 64 * SORT_KEEP) hipLaunchKernelGGL(moe_place_kernel<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(moe_place_kernel<false>, grid, block, 0, s, a);
    return (int)hipGetLastError();
}

// ---------------------------------------------------------------- rows without a slot

// Waves at the end of a launch write zeros to the rows that no slot fills.  Wave w of `waves` looks at the rows w,
// w + waves, ..., up to 64 at a time, so that a long stretch of such rows (behind the last group) is shared by all.
template <class F>
__device__ __forceinline__ void for_empty_rows(const int32_t* source, int64_t rows, int64_t slots, int64_t wave,
                                               int64_t waves, F&& zero) {
    const int lane = threadIdx.x & 63;
    for (int64_t r0 = wave; r0 < rows; r0 += 64 * waves) {
        const int64_t r = r0 + lane * waves;
        bool empty = false;
        if (r < rows) {
            const int32_t i = source[r];
            empty = i < 0 || i >= slots;
        }
        for (uint64_t m = __ballot(empty); m != 0; m &= m - 1) zero(r0 + __builtin_ctzll(m) * waves);
    }
}

// ---------------------------------------------------------------- gather

constexpr int MOE_THREADS = 256, MOE_WAVES = MOE_THREADS / 64;

struct MoeSlots {
    const int32_t* positions;   // [T][k]
    const int32_t* source;      // [rows]
    int64_t T;
    int k;
    int64_t rows;
};

// The rows of token t's slots, k <= 64 of them: lane j fetches slot j's, all in one trip to memory.  Fetched one after
// another (for_slots with FEW false), each waits for a trip of its own; a full chip does not mind, and MXFP8 rows, and
// a combination of few, do better so paced.  us with lanes and one after another: 64 tokens x 8 of 4096, MXFP8 without
// padding 4.2 and 5.1, combination 4.2 and 6.6; MXFP8 8192 x 8 of 2048 31.0 and 28.8, combination 16384 x 2 of 4096 64.7
// and 62.5, 8192 x 8 of 2048 52.1 and 53.4.
struct TokenRows {
    int32_t p;
    uint64_t left;   // slots that have a row, in ascending order
    __device__ __forceinline__ TokenRows(const MoeSlots& s, int64_t t) {
        const int lane = threadIdx.x & 63;
        p = lane < s.k ? s.positions[t * s.k + lane] : -1;
        left = __ballot(p >= 0 && p < s.rows);
    }
    __device__ __forceinline__ int slot() const { return __builtin_ctzll(left); }
    __device__ __forceinline__ int64_t row() const { return __builtin_amdgcn_readlane(p, slot()); }
    __device__ __forceinline__ void next() { left &= left - 1; }
};

static bool few_tokens(int64_t waves) { return waves < 2048; }   // eight for each CU

// Calls body(slot, row) for token t's slots that have a row, in ascending order.
template <bool FEW, class F>
__device__ __forceinline__ void for_slots(const MoeSlots& s, int64_t t, F&& body) {
    if constexpr (FEW) {
        for (TokenRows rows(s, t); rows.left; rows.next()) body(rows.slot(), rows.row());
    } else {
        for (int j = 0; j < s.k; ++j) {
            const int32_t r = s.positions[t * s.k + j];
            if (r >= 0 && r < s.rows) body(j, (int64_t)r);
        }
    }
}

// Stores of 16 bytes; with NT past the caches, for rows that they could not hold until somebody reads them: half of the
// memory-side cache or more, in rows of whole 128-byte lines (a line that two rows share would be written twice: 45 us
// instead of 34 for MXFP8 rows of 2080 bytes).  us with and without: gather of 402 MB 68 and 74, the combination's
// backward of 671 MB 118 and 121, of 1208 MB with fp32 outputs 228 and 236; the combination, which writes in order, 63.6
// and 63.0, has none.
template <bool NT>
__device__ __forceinline__ void put(void* p, const uint4 v) {
    if constexpr (NT) __builtin_nontemporal_store(u32v4{v.x, v.y, v.z, v.w}, (u32v4*)p);
    else *(uint4*)p = v;
}

static bool past_caches(int64_t rows, int64_t row_bytes) {
    return row_bytes % 128 == 0 && rows * row_bytes >= (int64_t)128 << 20;
}

struct GatherArgs {
    const uint16_t* x;
    int64_t ldx, H;
    MoeSlots s;
    unsigned token_groups;   // workgroups of the tokens; the others look for rows without a slot
    void* out;               // bf16 rows, or codes
    uint8_t* scales;
    float* s_enc;
};

// A token's row is read once and written k times.  A wave takes 512 U elements of a token.
template <int U, bool NT>
__global__ __launch_bounds__(MOE_THREADS) void moe_gather_kernel(GatherArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    uint16_t* out = (uint16_t*)a.out;
    if (blockIdx.x >= a.token_groups) {
        const int64_t w = (int64_t)(blockIdx.x - a.token_groups) * MOE_WAVES + wave;
        for_empty_rows(a.s.source, a.s.rows, a.s.T * a.s.k, w, (int64_t)(gridDim.x - a.token_groups) * MOE_WAVES, [&](int64_t r) {
            for (int64_t c = 8 * lane; c < a.H; c += 512) put<NT>(out + r * a.H + c, make_uint4(0, 0, 0, 0));
        });
        return;
    }
    const int64_t pieces = (a.H + 512 * U - 1) / (512 * U);
    const int64_t u = (int64_t)blockIdx.x * MOE_WAVES + wave, t = u / pieces, c0 = (u % pieces) * (512 * U) + 8 * lane;
    if (t >= a.s.T) return;
    TokenRows rows(a.s, t);
    uint4 v[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
        if (c0 + 512 * i < a.H) v[i] = load16_stream(a.x + t * a.ldx + c0 + 512 * i);
    for (; rows.left; rows.next()) {
        const int64_t r = rows.row();
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (c0 + 512 * i < a.H) put<NT>(out + r * a.H + c0 + 512 * i, v[i]);
    }
}

// Workgroups for the rows without a slot: a wave for 4 rows up to one workgroup a CU, then for 64 up to four.  us with a
// wave for 64 rows throughout, where most rows are padding: 4 tokens x 8 of 128 experts, bf16 4096 wide, 22 and now 4;
// 64 x 8 MXFP8 16.8 and 5.7.  Of many rows few are empty, and every workgroup that looks for them costs: 66 thousand of
// MXFP8 34.1, with 1024 workgroups 35.9.
static unsigned empty_groups(int64_t rows) {
    auto groups = [&](int64_t each, int64_t most) {
        const int64_t g = (rows + each * MOE_WAVES - 1) / (each * MOE_WAVES);
        return (unsigned)(g < 1 ? 1 : g > most ? most : g);
    };
    const unsigned few = groups(4, 256), many = groups(64, 1024);
    return few > many ? few : many;
}

constexpr int GATHER_U = 4;   // vectors of a lane: 2 and 8 within 2 %
static unsigned gather_groups(int64_t T, int64_t H) {
    return (unsigned)((T * ((H + 512 * GATHER_U - 1) / (512 * GATHER_U)) + MOE_WAVES - 1) / MOE_WAVES);
}

int launch_moe_gather(const void* x, int64_t ldx, int64_t T, int64_t k, int64_t H, const int32_t* positions,
                      const int32_t* source, int64_t rows, void* out, void* hip_stream) {
    if (rows == 0 || H == 0) return 0;
    const GatherArgs a{(const uint16_t*)x, ldx, H, {positions, source, T, (int)k, rows}, gather_groups(T, H), out, nullptr, nullptr};
    const dim3 grid(a.token_groups + empty_groups(rows)), block(MOE_THREADS);
    if (past_caches(rows, H * 2)) hipLaunchKernelGGL((moe_gather_kernel<GATHER_U, true>), grid, block, 0, (hipStream_t)hip_stream, a);
    else hipLaunchKernelGGL((moe_gather_kernel<GATHER_U, false>), grid, block, 0, (hipStream_t)hip_stream, a);
    return (int)hipGetLastError();
}

__device__ __forceinline__ float max8(const float v[8]) {
    float m = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = __builtin_fmaxf(m, __builtin_fabsf(v[e]));
    return m;
}

// The MXFP8 codes and scale byte of a lane's 8 elements of a block of 32, which 4 lanes share.  Each block is encoded as
// its own amax asks: a value that is not finite becomes NaN whatever the wave's other blocks hold.
__device__ __forceinline__ void mx_row_unit(const uint4 q, uint2& w, uint32_t& sb) {
    const uint32_t p[4] = {q.x, q.y, q.z, q.w};
    const uint32_t M = mx_quad_amax(p);
    const bool small = (M & 0xFFFFu) < MX_PACKED_LEAST;
    mx_encode_packed(p, small ? 0x3F803F80u : M, w.x, w.y, sb);
    if (__ballot(small) == 0) return;
    float v[8];
    unpack_bf16x8(q, v);
    if (small) {   // the scale byte is 0: amax below 2^-118, zero among them
        const float inv = mx_inv_scale(0);
        w = make_uint2(e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                       e4m3_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
        if ((M & 0xFFFFu) == 0) w = make_uint2(0, 0);   // -0 among them
        sb = 0;
    }
}

// MXFP8: a token is cast once, and its codes and scales written k times.  A lane holds a quarter of a block of 32.
template <int U, bool FEW>
__global__ __launch_bounds__(MOE_THREADS) void moe_gather_mxfp8_kernel(GatherArgs a) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    uint8_t* codes = (uint8_t*)a.out;
    const int64_t S = a.H / 32;
    if (blockIdx.x >= a.token_groups) {
        const int64_t w = (int64_t)(blockIdx.x - a.token_groups) * MOE_WAVES + wave;
        for_empty_rows(a.s.source, a.s.rows, a.s.T * a.s.k, w, (int64_t)(gridDim.x - a.token_groups) * MOE_WAVES, [&](int64_t r) {
            for (int64_t c = 16 * lane; c < a.H; c += 1024) *(uint4*)(codes + r * a.H + c) = make_uint4(0, 0, 0, 0);
            for (int64_t b = lane; b < S; b += 64) a.scales[r * S + b] = 0;
        });
        return;
    }
    const int64_t pieces = (a.H + 512 * U - 1) / (512 * U);
    const int64_t u = (int64_t)blockIdx.x * MOE_WAVES + wave, t = u / pieces, c0 = (u % pieces) * (512 * U) + 8 * lane;
    if (t >= a.s.T) return;
    uint4 q[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        q[i] = make_uint4(0, 0, 0, 0);
        if (c0 + 512 * i < a.H) q[i] = load16_stream(a.x + t * a.ldx + c0 + 512 * i);
    }
    uint2 w[U];
    uint32_t sb[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        mx_row_unit(q[i], w[i], sb[i]);
    }
    for_slots<FEW>(a.s, t, [&](int, int64_t r) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t c = c0 + 512 * i;
            if (c >= a.H) continue;
            *(uint2*)(codes + r * a.H + c) = w[i];
            if ((lane & 3) == 0) a.scales[r * S + c / 32] = (uint8_t)sb[i];
        }
    });
}

int launch_moe_gather_mxfp8(const void* x, int64_t ldx, int64_t T, int64_t k, int64_t H, const int32_t* positions,
                            const int32_t* source, int64_t rows, uint8_t* codes, uint8_t* scales, void* hip_stream) {
    if (rows == 0 || H == 0) return 0;
    const GatherArgs a{(const uint16_t*)x, ldx, H, {positions, source, T, (int)k, rows}, gather_groups(T, H), codes, scales, nullptr};
    const dim3 grid(a.token_groups + empty_groups(rows)), block(MOE_THREADS);
    if (few_tokens((int64_t)a.token_groups * MOE_WAVES))
        hipLaunchKernelGGL((moe_gather_mxfp8_kernel<GATHER_U, true>), grid, block, 0, (hipStream_t)hip_stream, a);
    else
        hipLaunchKernelGGL((moe_gather_mxfp8_kernel<GATHER_U, false>), grid, block, 0, (hipStream_t)hip_stream, a);
    return (int)hipGetLastError();
}

// Row-scaled NVFP4: W waves take a token, whose largest magnitude comes first; a lane holds whole blocks of 16.  U
// blocks a lane stay in registers in between; longer rows (W = 4 only) are read twice.
template <int U, int W>
__global__ __launch_bounds__(MOE_THREADS) void moe_gather_nvfp4_kernel(GatherArgs a) {
    __shared__ float red[MOE_WAVES];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    uint8_t* codes = (uint8_t*)a.out;
    const int64_t C = a.H / 2, S = a.H / 16;
    if (blockIdx.x >= a.token_groups) {
        const int64_t w = (int64_t)(blockIdx.x - a.token_groups) * MOE_WAVES + wave;
        for_empty_rows(a.s.source, a.s.rows, a.s.T * a.s.k, w, (int64_t)(gridDim.x - a.token_groups) * MOE_WAVES, [&](int64_t r) {
            for (int64_t b = lane; b < S; b += 64) {
                *(uint2*)(codes + r * C + 8 * b) = make_uint2(0, 0);
                a.scales[r * S + b] = 0;
            }
            if (lane == 0) a.s_enc[r] = 1.0f;
        });
        return;
    }
    const int64_t t = W == 1 ? (int64_t)blockIdx.x * MOE_WAVES + wave : (int64_t)blockIdx.x;
    if (W == 1 && t >= a.s.T) return;
    const TokenRows all(a.s, t);
    const int first = W == 1 ? lane : (int)threadIdx.x;   // the thread's first block; its others 64 W apart
    const uint16_t* x = a.x + t * a.ldx;
    const bool one = W == 1 || S <= 64 * U * W;
    uint4 q[U][2];
    float m = 0.0f;
    auto load = [&](int64_t b0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int64_t b = b0 + first + 64 * W * i;
            q[i][0] = q[i][1] = make_uint4(0, 0, 0, 0);
            if (b < S) {
                q[i][0] = *(const uint4*)(x + 16 * b);
                q[i][1] = *(const uint4*)(x + 16 * b + 8);
            }
        }
    };
    auto values = [&](int i, float v[16]) {
        unpack_bf16x8(q[i][0], v);
        unpack_bf16x8(q[i][1], v + 8);
        return __builtin_fmaxf(max8(v), max8(v + 8));
    };
    for (int64_t b0 = 0; b0 < S; b0 += 64 * U * W) {
        load(b0);
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float v[16];
            m = __builtin_fmaxf(m, values(i, v));
        }
    }
    m = wave_max(m);
    if constexpr (W > 1) {
        if (lane == 0) red[wave] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < W; ++w) m = __builtin_fmaxf(m, red[w]);
    }
    const float Se = nvfp4_tensor_scale(m);
    for (int64_t b0 = 0; b0 < S; b0 += 64 * U * W) {
        if (!one) load(b0);
        uint32_t w[U][2], sb[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            float v[16];
            const float bm = values(i, v);
            sb[i] = encode_block<16, false, false>(v, bm, Se, nullptr, 0, 0, 0, 0, w[i]);
        }
        for (TokenRows rows = all; rows.left; rows.next()) {
            const int64_t r = rows.row();
            if (b0 == 0 && first == 0) a.s_enc[r] = Se;
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const int64_t b = b0 + first + 64 * W * i;
                if (b >= S) continue;
                *(uint2*)(codes + r * C + 8 * b) = make_uint2(w[i][0], w[i][1]);
                a.scales[r * S + b] = (uint8_t)sb[i];
            }
        }
    }
}

// Rows of width 0 have a scale all the same, that of a row without a value above 0.
__global__ __launch_bounds__(MOE_THREADS) void moe_gather_scales_kernel(float* s_enc, int64_t rows) {
    const int64_t r = (int64_t)blockIdx.x * MOE_THREADS + threadIdx.x;
    if (r < rows) s_enc[r] = nvfp4_tensor_scale(0.0f);
}

int launch_moe_gather_nvfp4(const void* x, int64_t ldx, int64_t T, int64_t k, int64_t H, const int32_t* positions,
                            const int32_t* source, int64_t rows, uint8_t* codes, uint8_t* scales, float* s_enc,
                            void* hip_stream) {
    if (rows == 0) return 0;
    hipStream_t s = (hipStream_t)hip_stream;
    if (H == 0) {
        hipLaunchKernelGGL(moe_gather_scales_kernel, dim3((unsigned)((rows + MOE_THREADS - 1) / MOE_THREADS)), dim3(MOE_THREADS), 0, s, s_enc, rows);
        return (int)hipGetLastError();
    }
    // a wave a token where that leaves every CU eight of them, else a workgroup
    const bool wave = T >= 2048 && H <= 4096;
    const GatherArgs a{(const uint16_t*)x, ldx, H, {positions, source, T, (int)k, rows},
                       (unsigned)(wave ? (T + MOE_WAVES - 1) / MOE_WAVES : T), codes, scales, s_enc};
    const dim3 grid(a.token_groups + empty_groups(rows)), block(MOE_THREADS);
    if (wave && H <= 2048) hipLaunchKernelGGL((moe_gather_nvfp4_kernel<2, 1>), grid, block, 0, s, a);
    else if (wave) hipLaunchKernelGGL((moe_gather_nvfp4_kernel<4, 1>), grid, block, 0, s, a);
    else if (H <= 4096) hipLaunchKernelGGL((moe_gather_nvfp4_kernel<1, 4>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((moe_gather_nvfp4_kernel<2, 4>), grid, block, 0, s, a);
    return (int)hipGetLastError();
}

// ---------------------------------------------------------------- combine

// A lane's part of 64 lanes' piece of a row: 16 bytes of the experts' outputs, 8 bf16 or 4 fp32 values, so that the
// lanes of every access are neighbours.
template <bool F32>
struct Piece {
    static constexpr int N = F32 ? 4 : 8;      // values of a lane
    static constexpr int ALL = 64 * N;         // of the wave
    uint4 q;
    __device__ __forceinline__ void load(const void* y, int64_t at) {
        q = load16_stream((const uint8_t*)y + at * (F32 ? 4 : 2));
    }
    __device__ __forceinline__ void values(float (&v)[N]) const {
        if constexpr (F32) {
            v[0] = __uint_as_float(q.x); v[1] = __uint_as_float(q.y);
            v[2] = __uint_as_float(q.z); v[3] = __uint_as_float(q.w);
        } else {
            unpack_bf16x8(q, v);
        }
    }
};

// N = 4 or 8 bf16 values.
template <int N>
__device__ __forceinline__ void load_bf16(const uint16_t* p, float (&v)[N]) {
    if constexpr (N == 8) {
        unpack_bf16x8(*(const uint4*)p, v);
    } else {
        const uint2 q = *(const uint2*)p;
        v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x);
        v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
    }
}

template <bool F32, bool NT, int N>
__device__ __forceinline__ void store_row(void* y, int64_t at, const float (&v)[N]) {
    if constexpr (F32) {
#pragma unroll
        for (int e = 0; e < N; e += 4)
            put<NT>((float*)y + at + e, make_uint4(__float_as_uint(v[e]), __float_as_uint(v[e + 1]), __float_as_uint(v[e + 2]),
                                                   __float_as_uint(v[e + 3])));
    } else if constexpr (N == 8) {
        put<NT>((uint16_t*)y + at,
                make_uint4(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]), bf16x2_rne(v[4], v[5]), bf16x2_rne(v[6], v[7])));
    } else {
        *(uint2*)((uint16_t*)y + at) = make_uint2(bf16x2_rne(v[0], v[1]), bf16x2_rne(v[2], v[3]));
    }
}

struct CombineArgs {
    const void* y;
    int64_t H;
    MoeSlots s;
    const float* weights;   // [T][k], or none
    void* out;
};

// Sums in fp32 over j in ascending order, one rounding to the output's type.
template <bool YF32, bool OF32, bool FEW>
__global__ __launch_bounds__(MOE_THREADS) void moe_combine_kernel(CombineArgs a) {
    typedef Piece<YF32> P;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int64_t pieces = (a.H + P::ALL - 1) / P::ALL, group = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
    const int64_t u = group * MOE_WAVES + wave, t = u / pieces, c = (u % pieces) * P::ALL + P::N * lane;
    if (t >= a.s.T) return;
    float acc[P::N] = {};
    auto add = [&](float w, const P& q) {
        float y[P::N];
        q.values(y);
#pragma unroll
        for (int e = 0; e < P::N; ++e) acc[e] = __builtin_fmaf(w, y[e], acc[e]);
    };
    if constexpr (FEW) {
        constexpr int G = 4;   // rows in flight
        TokenRows rows(a.s, t);
        const float weight = a.weights && lane < a.s.k ? a.weights[t * a.s.k + lane] : 1.0f;   // of slot `lane`
        while (rows.left) {
            float w[G];
            P q[G];
            int n = 0;
#pragma unroll
            for (int u = 0; u < G; ++u)
                if (rows.left) {
                    w[u] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), rows.slot()));
                    if (c < a.H) q[u].load(a.y, rows.row() * a.H + c);
                    rows.next();
                    ++n;
                }
#pragma unroll
            for (int u = 0; u < G; ++u)
                if (u < n) add(w[u], q[u]);
        }
        if (c >= a.H) return;
    } else {
        if (c >= a.H) return;
        for_slots<false>(a.s, t, [&](int j, int64_t r) {
            P q;
            q.load(a.y, r * a.H + c);
            add(a.weights ? a.weights[t * a.s.k + j] : 1.0f, q);
        });
    }
    store_row<OF32, false>(a.out, t * a.H + c, acc);
}

int launch_moe_combine(const void* y, int y_f32, int64_t T, int64_t k, int64_t H, const int32_t* positions, int64_t rows,
                       const float* weights, void* out, int out_f32, void* hip_stream) {
    if (T == 0 || H == 0) return 0;
    hipStream_t s = (hipStream_t)hip_stream;
    const CombineArgs a{y, H, {positions, nullptr, T, (int)k, rows}, weights, out};
    const int64_t width = y_f32 ? Piece<true>::ALL : Piece<false>::ALL, waves = T * ((H + width - 1) / width);
    const int64_t groups = (waves + MOE_WAVES - 1) / MOE_WAVES;   // fp32 rows: up to 2^24, a thread more than x holds
    const unsigned high = groups > (int64_t)1 << 23 ? 2 : 1;
    const dim3 grid((unsigned)((groups + high - 1) / high), high), block(MOE_THREADS);
    auto launch = [&](auto few_c) {
        constexpr bool FEW = decltype(few_c)::value;
        if (y_f32 && out_f32) hipLaunchKernelGGL((moe_combine_kernel<true, true, FEW>), grid, block, 0, s, a);
        else if (y_f32) hipLaunchKernelGGL((moe_combine_kernel<true, false, FEW>), grid, block, 0, s, a);
        else if (out_f32) hipLaunchKernelGGL((moe_combine_kernel<false, true, FEW>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((moe_combine_kernel<false, false, FEW>), grid, block, 0, s, a);
    };
    if (few_tokens(waves)) launch(std::true_type{});
    else launch(std::false_type{});
    return (int)hipGetLastError();
}

struct CombineBwdArgs {
    const uint16_t* dout;
    const void* y;
    int64_t H;
    MoeSlots s;
    const float* weights;
    void* dy;
    float* dweights;
    unsigned token_groups;
};

// A wave takes a slot: the token's row of dout (which the waves of its other slots read about the same time, so that it
// comes from memory once) with the slot's row of y, U pieces of it at a time.
template <bool YF32, int U, bool NT>
__global__ __launch_bounds__(MOE_THREADS) void moe_combine_backward_kernel(CombineBwdArgs a) {
    typedef Piece<YF32> P;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    if (blockIdx.x >= a.token_groups) {
        const int64_t w = (int64_t)(blockIdx.x - a.token_groups) * MOE_WAVES + wave;
        for_empty_rows(a.s.source, a.s.rows, a.s.T * a.s.k, w, (int64_t)(gridDim.x - a.token_groups) * MOE_WAVES, [&](int64_t r) {
            const float zero[P::N] = {};
            for (int64_t c = P::N * lane; c < a.H; c += P::ALL) store_row<YF32, NT>(a.dy, r * a.H + c, zero);
        });
        return;
    }
    const int64_t i = (int64_t)blockIdx.x * MOE_WAVES + wave;
    if (i >= a.s.T * a.s.k) return;
    const int64_t t = i / a.s.k;
    const int32_t r = a.s.positions[i];
    if (r < 0 || r >= a.s.rows) {
        if (lane == 0) a.dweights[i] = 0.0f;
        return;
    }
    const float w = a.weights[i];
    float dot = 0.0f;
    for (int64_t c0 = P::N * lane; c0 < a.H; c0 += P::ALL * U) {
        float d[U][P::N];
        P q[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + P::ALL * u < a.H) {
                q[u].load(a.y, (int64_t)r * a.H + c0 + P::ALL * u);
                load_bf16(a.dout + t * a.H + c0 + P::ALL * u, d[u]);
            }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (c0 + P::ALL * u < a.H) {
                float v[P::N];
                q[u].values(v);
#pragma unroll
                for (int e = 0; e < P::N; ++e) {
                    dot = __builtin_fmaf(d[u][e], v[e], dot);
                    d[u][e] = w * d[u][e];
                }
                store_row<YF32, NT>(a.dy, (int64_t)r * a.H + c0 + P::ALL * u, d[u]);
            }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) dot += __shfl_xor(dot, o);
    if (lane == 0) a.dweights[i] = dot;
}

int launch_moe_combine_backward(const void* dout, const void* y, int y_f32, int64_t T, int64_t k, int64_t H,
                                const int32_t* positions, const int32_t* source, int64_t rows, const float* weights,
                                void* dy, float* dweights, void* hip_stream) {
    if (T * k == 0 && rows == 0) return 0;
    hipStream_t s = (hipStream_t)hip_stream;
    const unsigned tg = (unsigned)((T * k + MOE_WAVES - 1) / MOE_WAVES);
    const CombineBwdArgs a{(const uint16_t*)dout, y, H, {positions, source, T, (int)k, rows}, weights, dy, dweights, tg};
    const dim3 grid(tg + empty_groups(rows)), block(MOE_THREADS);
    auto launch = [&](auto nt_c) {
        constexpr bool NT = decltype(nt_c)::value;
        if (y_f32) hipLaunchKernelGGL((moe_combine_backward_kernel<true, 2, NT>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((moe_combine_backward_kernel<false, 4, NT>), grid, block, 0, s, a);
    };
    if (past_caches(rows, H * (y_f32 ? 4 : 2))) launch(std::true_type{});
    else launch(std::false_type{});
    return (int)hipGetLastError();
}

}  // namespace bsq
