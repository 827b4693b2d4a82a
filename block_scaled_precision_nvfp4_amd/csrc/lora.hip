// lora.hip -- low-rank adapters beside a projection, each token with its own: out[m] = y[m] + s_a (x[m] A_a^T) B_a^T with a
// the token's adapter, A [L][r][K], B [L][N][r].
//
// Two kernels: the down products t[m] = x[m] A_a^T into the caller's workspace, then the up products onto y.
// Few tokens are taken one by one, whatever their adapters; beside NVFP4 weights, their down products go along with
// the weights' product (matvec.hip).  Many go in tiles of 16, the rows of a matrix instruction; a tile's adapters are
// taken one after another, each over all 16 rows, and a row keeps the result of its own.  Rows do not mix, so a
// NaN stays with its token, or its adapter's tokens.
//
// Bound by memory where tokens are many (x once, y once each way), by latency where they are few.  us in a graph, states
// rotating through 800 MB: 16 tokens of 16 adapters, rank 16, 4096 x 4096 6.4; 64 of one adapter, rank 64, 11.1;
// 1024 in runs, rank 16, 14336 x 4096 30; 4096 in runs of 8 adapters, rank 64, 4096 x 4096 39 (down 16, up 24; its
// bytes alone take 23 at the rate of a large copy), with K 14336 65, tokens of the same 8 adapters
// shuffled 144: every tile then has most of them.
#include "launch.hpp"
#include "lora.hpp"

namespace bsq {

typedef float floatx4 __attribute__((ext_vector_type(4)));

constexpr int LORA_TOKENS = 16;

// The ids of a tile's adapters: lane i holds token i % 16's, -1 for none.
__device__ __forceinline__ int lora_ids(const LoraArgs& a, int64_t m0) {
    const int64_t m = m0 + (threadIdx.x & 15);
    const int id = m < a.M ? a.adapters[m] : -1;
    return id >= 0 && id < a.L ? id : -1;
}

// Calls body(adapter) for the tile's adapters number first, first + step, ... in the order of their first tokens.
template <class F>
__device__ __forceinline__ void for_adapters(int ids, int first, int step, F&& body) {
    uint64_t left = __ballot(ids >= 0) & 0xFFFFu;
    for (int n = 0; left != 0; ++n) {
        const int id = __builtin_amdgcn_readlane(ids, __builtin_ctzll(left));
        left &= ~__ballot(ids == id);
        if (n >= first && (n - first) % step == 0) body(id);
    }
}

// t of a tile: blockIdx.x tile, .y which of its adapters, .z 16 NR ranks.  The waves share K, 64 elements (a
// 128-byte line) of every row at a time.  A wave reads whole lines, 8 lanes each, and turns them to the matrix
// instruction's order through LDS of its own: read in that order, neighbouring lanes would touch 16 lines, 16 bytes
// of each, at a quarter of the rate (25 us instead of 17).  D pieces are in flight in registers.  The waves' sums are
// joined in LDS, and go out as the up products' fragments.
constexpr int LORA_PITCH = 144;   // bytes between rows in LDS: the fragments' reads cover all banks
constexpr int lora_waves(int nr) { return nr == 4 ? 8 : 16; }

// Orders a wave's own accesses to LDS, which the hardware runs as they come, for the compiler.
__device__ __forceinline__ void lora_wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int NR>
__global__ __launch_bounds__(64 * lora_waves(NR)) void lora_down_kernel(LoraArgs a) {
    constexpr int W = lora_waves(NR), D = NR == 1 ? 4 : NR == 2 ? 2 : 1, ROWS = LORA_TOKENS * (NR + 1);
    static_assert(W * NR * LORA_TOKENS * 17 * 4 <= W * ROWS * LORA_PITCH, "the join takes the rows' place");
    __shared__ __attribute__((aligned(16))) uint8_t lds[W * ROWS * LORA_PITCH];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int r16 = lane & 15, g = lane >> 4, row8 = lane >> 3, k8 = 8 * (lane & 7);
    // neighbouring tiles, which mostly share an adapter, to one XCD (workgroups go to the 8 XCDs in turn)
    const unsigned per = gridDim.x / 8, tile = blockIdx.x < per * 8 ? blockIdx.x % 8 * per + blockIdx.x / 8 : blockIdx.x;
    const int64_t m0 = (int64_t)tile * LORA_TOKENS;
    const int rank0 = blockIdx.z * 16 * NR, K = (int)a.K, pieces = (K + 63) / 64;
    const int ids = lora_ids(a, m0);
    // tokens that no other workgroup reads pass the caches by, which A has for itself: 4096 tokens of 14336, rank 64, 70 -> 64 us
    const bool once = gridDim.y == 1 && gridDim.z == 1;
    uint8_t* mine = lds + wave * ROWS * LORA_PITCH;
    for_adapters(ids, blockIdx.y, gridDim.y, [&](int id) {
        const uint32_t rows = (uint32_t)__ballot(ids == id) & 0xFFFFu;   // the tile's tokens with this adapter
        // a lane's rows: tokens row8 and 8 + row8, ranks rank0 + 8 i + row8.  In the place of a token with another
        // adapter and of a rank past r, whose results nobody takes, one that is there stands.
        const uint16_t* from[2 * (NR + 1)];
#pragma unroll
        for (int i = 0; i < 2 * (NR + 1); ++i) {
            const int token = 8 * i + row8, rank = rank0 + 8 * (i - 2) + row8;
            from[i] = k8 + (i < 2 ? a.x + (m0 + ((rows >> token) & 1 ? token : __builtin_ctz(rows))) * a.ldx
                                  : a.a + ((int64_t)id * a.r + (rank < a.r ? rank : a.r - 1)) * a.K);
        }
        uint4 v[D][2 * (NR + 1)];
        auto load = [&](int d, int c) {
            if (64 * (c + 1) <= K) {
#pragma unroll
                for (int i = 0; i < 2 * (NR + 1); ++i)
                    v[d][i] = i < 2 && once ? load16_stream(from[i] + 64 * c) : *(const uint4*)(from[i] + 64 * c);
            } else {   // the piece that K ends in
#pragma unroll
                for (int i = 0; i < 2 * (NR + 1); ++i) {
                    v[d][i] = make_uint4(0, 0, 0, 0);
                    if (64 * c + k8 < K) v[d][i] = *(const uint4*)(from[i] + 64 * c);
                }
            }
        };
        floatx4 acc[NR];
#pragma unroll
        for (int n = 0; n < NR; ++n) acc[n] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
        auto use = [&](int d) {
#pragma unroll
            for (int i = 0; i < 2 * (NR + 1); ++i) *(uint4*)(mine + (8 * i + row8) * LORA_PITCH + 2 * k8) = v[d][i];
            lora_wave_fence();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint8_t* f = mine + r16 * LORA_PITCH + 32 * g + 16 * h;
                const bf16x8_t xv = *(const bf16x8_t*)f;
#pragma unroll
                for (int n = 0; n < NR; ++n)
                    acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, *(const bf16x8_t*)(f + 16 * (n + 1) * LORA_PITCH),
                                                                     acc[n], 0, 0, 0);
            }
            lora_wave_fence();
        };
        const int count = pieces > wave ? (pieces - wave - 1) / W + 1 : 0;   // pieces wave, wave + W, ...
#pragma unroll
        for (int d = 0; d < D; ++d)
            if (d < count) load(d, wave + d * W);
        for (int n = 0; n < count; n += D)
#pragma unroll
            for (int d = 0; d < D; ++d)
                if (n + d < count) {
                    use(d);
                    if (n + d + D < count) load(d, wave + (n + d + D) * W);
                }
        __syncthreads();
        float* red = (float*)lds;   // [wave][NR][16][17]
#pragma unroll
        for (int n = 0; n < NR; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) red[((wave * NR + n) * LORA_TOKENS + 4 * g + i) * 17 + r16] = acc[n][i];
        __syncthreads();
        for (int i = threadIdx.x; i < LORA_TOKENS * 16 * NR; i += 64 * W) {
            const int m = i / (16 * NR), n = i / 16 % NR, q = i % 16, rank = rank0 + 16 * n + q;
            if (!((rows >> m) & 1)) continue;
            float t = 0.0f;
#pragma unroll
            for (int u = 0; u < W; ++u) t += red[((u * NR + n) * LORA_TOKENS + m) * 17 + q];
            if (rank >= a.r) continue;
            uint16_t p[3];
            lora_split(t, p);
            uint16_t* at = (uint16_t*)a.t + ((int64_t)tile * lora_steps(a.r) + rank / 32) * 3 * 512 + (m + 16 * (rank / 8 % 4)) * 8 + rank % 8;
            at[0] = p[0];
            at[512] = p[1];
            at[1024] = p[2];
        }
        __syncthreads();   // before the next adapter's rows
    });
}

template <bool F32>
__device__ __forceinline__ float lora_y(const LoraArgs& a, int64_t m, int64_t n) {
    if constexpr (F32) return ((const float*)a.y)[m * a.ldy + n];
    else return __uint_as_float((uint32_t)((const uint16_t*)a.y)[m * a.ldy + n] << 16);
}

template <bool F32>
__device__ __forceinline__ void lora_store(const LoraArgs& a, int64_t m, int64_t n, float v) {
    if constexpr (F32) ((float*)a.out)[m * a.ldo + n] = v;
    else ((uint16_t*)a.out)[m * a.ldo + n] = (uint16_t)bf16x2_rne(v, 0.0f);
}

// The up products of a tile of 16 tokens per wave by `chunks` times 64 columns, one after another.  The workgroup's waves
// take neighbouring tiles, which mostly share an adapter: its 64 rows of B come through LDS, whole lines at a time,
// for all of them, the next ones (and y's) asked for before the present ones are used.  t comes as the matrix
// instruction's fragments, in three bf16 parts (lora_split).  Column r16 of block b stands for column 4 r16 + b,
// so that a lane ends with 4 adjacent columns of each of 4 tokens (4 g + i) and 16 lanes read and write 128 (or 256)
// adjacent bytes of y.
constexpr int LORA_UP_WAVES = 4, LORA_COLS = 64;

// Four adjacent values of y or out, aligned to a value only (odd row lengths), in one access all the same: 4096 x 4097 x
// 4096, rank 64, in 46 us where single values took 82; 4096 columns 39.
template <bool F32>
struct __attribute__((packed, aligned(F32 ? 4 : 2))) LoraY {
    uint32_t w[F32 ? 4 : 2];
    __device__ __forceinline__ void values(float (&f)[4]) const {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = F32 ? __uint_as_float(w[i]) : i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
    }
};

__device__ __forceinline__ LoraY<true> lora_four(const float (&f)[4], std::true_type) {
    return {{__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3])}};
}
__device__ __forceinline__ LoraY<false> lora_four(const float (&f)[4], std::false_type) {
    return {{bf16x2_rne(f[0], f[1]), bf16x2_rne(f[2], f[3])}};
}

// YF, OF: y and out are fp32.  RS: steps of 32 ranks.  WHOLE: N is a multiple of 64.
template <bool YF, bool OF, int RS, bool WHOLE>
__global__ __launch_bounds__(64 * LORA_UP_WAVES) void lora_up_kernel(LoraArgs a, int chunks) {
    constexpr int PITCH = 64 * RS + 16;   // bytes between rows in LDS; the fragments' reads cover all banks
    constexpr int BV = RS;                // 16-byte pieces of B of a thread: 64 rows of 4 RS pieces for 256
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][LORA_COLS * PITCH];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int r16 = lane & 15, g = lane >> 4;
    const int64_t cols = (a.N + LORA_COLS - 1) / LORA_COLS, groups = (cols + chunks - 1) / chunks;
    const int64_t first = blockIdx.x % groups * chunks;
    const int last = (int)(cols - first < chunks ? cols - first : chunks);
    const int64_t tile0 = blockIdx.x / groups * LORA_UP_WAVES, m0 = (tile0 + wave) * LORA_TOKENS;
    typedef typename std::conditional<YF, float, uint16_t>::type item;
    typedef LoraY<YF> vec;
    const int steps = lora_steps(a.r), cpr = a.r / 8;    // 16-byte pieces of a row of B
    const int64_t ml = tile0 * LORA_TOKENS + lane;       // lane's of the workgroup's 64 tokens
    int all = ml < a.M ? a.adapters[ml] : -1;
    all = all >= 0 && all < a.L ? all : -1;
    bf16x8_t part[RS][3];
#pragma unroll
    for (int q = 0; q < RS; ++q)
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            part[q][p] = bf16x8_t{};   // past r nothing is written
            if (32 * q + 8 * g < a.r && m0 < a.M)
                part[q][p] = *(const bf16x8_t*)((const uint16_t*)a.t + (((tile0 + wave) * steps + q) * 3 + p) * 512 + 8 * lane);
        }
    auto column = [&](int c) { return (first + c) * LORA_COLS + 4 * r16; };
    vec v[4], vn[4];
    auto load_y = [&](int c, vec (&d)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (m0 + 4 * g + i >= a.M) continue;
            const item* y = (const item*)a.y + (m0 + 4 * g + i) * a.ldy + column(c);
            const int64_t n = a.N - column(c);   // columns from here on
            if (WHOLE || n >= 4) {
                d[i] = *(const vec*)y;
            } else if constexpr (YF) {
#pragma unroll
                for (int b = 0; b < 3; ++b) d[i].w[b] = b < n ? __float_as_uint(y[b]) : 0u;
            } else {
                d[i].w[0] = n > 0 ? y[0] : 0u;
                d[i].w[0] |= n > 1 ? (uint32_t)y[1] << 16 : 0u;
                d[i].w[1] = n > 2 ? y[2] : 0u;
            }
        }
    };
    int row[BV], piece[BV];   // of the thread's pieces of B
#pragma unroll
    for (int e = 0; e < BV; ++e) {
        const int at = (int)threadIdx.x + 256 * e;
        row[e] = at / cpr;
        piece[e] = at - row[e] * cpr;
    }
    uint4 wb[BV];
    auto load_b = [&](int c, int id) {
        const int64_t n0 = (first + c) * LORA_COLS;
#pragma unroll
        for (int e = 0; e < BV; ++e) {
            wb[e] = make_uint4(0, 0, 0, 0);
            if (row[e] < LORA_COLS && n0 + row[e] < a.N)
                wb[e] = *(const uint4*)(a.b + ((int64_t)id * a.N + n0 + row[e]) * a.r + 8 * piece[e]);
        }
    };
    load_y(0, v);
    int mine[4];   // the adapters of the lane's tokens of y
    float scale[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        mine[i] = __shfl(all, 16 * wave + 4 * g + i);
        scale[i] = a.scales && mine[i] >= 0 ? a.scales[mine[i]] : 1.0f;
    }
    const uint64_t some = __ballot(all >= 0);   // the same in every wave
    if (some == 0 && a.out == a.y) return;
    auto finish = [&](int c, const floatx4 (&add)[4]) {
        const int64_t c0 = column(c);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t m = m0 + 4 * g + i;
            const bool has = mine[i] >= 0;
            if (m >= a.M || (!has && a.out == a.y)) continue;
            float f[4];
            v[i].values(f);
            if (has)
#pragma unroll
                for (int b = 0; b < 4; ++b) f[b] = __builtin_fmaf(scale[i], add[i][b], f[b]);
            if (WHOLE || c0 + 4 <= a.N) {
                typedef typename std::conditional<OF, float, uint16_t>::type result;
                *(LoraY<OF>*)((result*)a.out + m * a.ldo + c0) = lora_four(f, std::integral_constant<bool, OF>{});
            } else {
#pragma unroll
                for (int b = 0; b < 3; ++b)
                    if (c0 + b < a.N) lora_store<OF>(a, m, c0 + b, f[b]);
            }
        }
    };
    floatx4 add[4] = {};
    if (some == 0) {   // no token has one: y goes over
        for (int c = 0; c < last; ++c) {
            if (c > 0) load_y(c, v);
            finish(c, add);
        }
        return;
    }
    // steps: the adapters of a chunk of columns, then the next chunk
    uint64_t left = some;
    int c = 0, id = __builtin_amdgcn_readlane(all, __builtin_ctzll(left)), buf = 0;
    load_b(0, id);
    while (true) {
        const uint64_t here = __ballot(all == id);
        left &= ~here;
        const bool ends = left == 0;   // the chunk's last step
        if (ends) left = some;
        const int next = __builtin_amdgcn_readlane(all, __builtin_ctzll(left)), nc = ends ? c + 1 : c;
#pragma unroll
        for (int e = 0; e < BV; ++e)   // block b's rows side by side
            if (row[e] < LORA_COLS) *(uint4*)(lds[buf] + ((row[e] & 3) * 16 + (row[e] >> 2)) * PITCH + 16 * piece[e]) = wb[e];
        if (nc < last) {
            load_b(nc, next);
            if (ends) load_y(nc, vn);
        }
        __syncthreads();
        if ((here >> (16 * wave)) & 0xFFFFu) {
            floatx4 acc[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) acc[b] = floatx4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int q = 0; q < RS; ++q) {
                bf16x8_t w[4] = {};
                if (32 * q + 8 * g < a.r)
#pragma unroll
                    for (int b = 0; b < 4; ++b) w[b] = *(const bf16x8_t*)(lds[buf] + (16 * b + r16) * PITCH + 64 * q + 16 * g);
#pragma unroll
                for (int p = 2; p >= 0; --p)   // four sums in turn: an instruction does not wait for the one before
#pragma unroll
                    for (int b = 0; b < 4; ++b) acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(part[q][p], w[b], acc[b], 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (mine[i] == id) add[i] = floatx4{acc[0][i], acc[1][i], acc[2][i], acc[3][i]};
        }
        if (ends) {
            finish(c, add);
            if (nc == last) return;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = vn[i];
        }
        c = nc;
        id = next;
        buf ^= 1;
    }
}

// Few tokens: a wave takes some columns of one, so that any mixture of adapters goes at once.  G lanes share a row of B,
// 16 bytes each, and 64 / G neighbouring rows are a load; the sums of I loads are then added up across the G lanes in
// halves, which leaves the lanes with a column each.  (A lane with a row of its own touches a line with each load.)  No
// more than 4 loads: a wave runs through its code once, and every line of that comes from memory too.  us, against a
// row for each lane: 64 tokens of 64 adapters, rank 64, 4096 x 4096, 19.1 and 25.6; one token, rank 256, 6.8 and 13.2 (7.6
// with 8 loads, 22 with 32).
constexpr int lora_few_loads(int lanes) { return lanes < 4 ? lanes : 4; }

// G: lanes of a row, a power of two, 8 G >= r.
template <bool YF, bool OF, int G>
__global__ __launch_bounds__(256) void lora_up_few_kernel(LoraArgs a) {
    constexpr int I = lora_few_loads(G), C = I * (64 / G);   // columns of a wave
    const int lane = threadIdx.x & 63, pos = lane & (G - 1), sub = lane / G;
    const int64_t m = blockIdx.y, n0 = ((int64_t)blockIdx.x * 4 + threadIdx.x / 64) * C, n = n0 + pos / (G / I) * (64 / G) + sub;
    const int id = a.adapters[m];
    const bool has = id >= 0 && id < a.L;
    if (n0 >= a.N || (!has && a.out == a.y)) return;
    float y = 0.0f;
    if (n < a.N) y = lora_y<YF>(a, m, n);
    if (has) {
        const bool in = 8 * pos < a.r;
        float t[8] = {};
        if (in) {
            const float4 t0 = *(const float4*)(a.t + m * a.r + 8 * pos), t1 = *(const float4*)(a.t + m * a.r + 8 * pos + 4);
            t[0] = t0.x; t[1] = t0.y; t[2] = t0.z; t[3] = t0.w;
            t[4] = t1.x; t[5] = t1.y; t[6] = t1.z; t[7] = t1.w;
        }
        const uint16_t* b = a.b + (int64_t)id * a.N * a.r + (in ? 8 * pos : 0);
        uint4 v[I];
#pragma unroll
        for (int i = 0; i < I; ++i) {   // of column n0 + i (64 / G) + sub, or the last one, whose sum nobody takes
            const int64_t c = n0 + i * (64 / G) + sub;
            v[i] = *(const uint4*)(b + (c < a.N ? c : a.N - 1) * a.r);
        }
        float s[I];
#pragma unroll
        for (int i = 0; i < I; ++i) {
            const uint4 q = in ? v[i] : make_uint4(0, 0, 0, 0);
            float w[8];
            unpack_bf16x8(q, w);
            s[i] = 0.0f;
#pragma unroll
            for (int e = 0; e < 8; ++e) s[i] = __builtin_fmaf(t[e], w[e], s[i]);
        }
#pragma unroll
        for (int h = G / 2; h > 0; h /= 2) {
            const int half = h * I / G;   // sums that a lane keeps
#pragma unroll
            for (int i = 0; i < half; ++i) {
                const bool high = pos & h;
                const float other = __shfl_xor(high ? s[i] : s[i + half], h);
                s[i] = (high ? s[i + half] : s[i]) + other;
            }
            if (half == 0) s[0] += __shfl_xor(s[0], h);
        }
        y = __builtin_fmaf(a.scales ? a.scales[id] : 1.0f, s[0], y);
    }
    if (n < a.N && pos % (G / I) == 0) lora_store<OF>(a, m, n, y);
}

__global__ __launch_bounds__(256) void lora_down_few_kernel(LoraArgs a, int rq) {
    lora_down_few(a, rq, (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6)));
}

int launch_lora_down_few(const LoraArgs& a, hipStream_t s) {
    const int rq = lora_few_rows(a.M, a.r);
    hipLaunchKernelGGL(lora_down_few_kernel, dim3((unsigned)((lora_few_units(a.M, a.r, rq) + 3) / 4)), dim3(256), 0, s, a, rq);
    return (int)hipGetLastError();
}

int launch_lora_down_many(const LoraArgs& a, hipStream_t s) {
    const int64_t tiles = (a.M + LORA_TOKENS - 1) / LORA_TOKENS;
    // 64 ranks a workgroup, which then reads x once, or fewer while that leaves CUs idle; and a workgroup for each
    // adapter that a tile may have while CUs are left even so.  us of the whole call with 64 ranks a workgroup and
    // by this rule, tokens x 4096 x 4096 in runs, rank 64: 128 tokens 16.6 and 12.6, 256 21.4 and 15.0, 1024
    // 24.7 and 18.8, 2048 29.2 and 24.5; 1024 tokens of 8 adapters shuffled, rank 32, 33 and 41.
    int nr = 4;
    while (nr > 1 && (16 * (nr / 2) >= a.r || tiles * ((a.r + 16 * nr - 1) / (16 * nr)) < 256)) nr /= 2;
    const int64_t z = (a.r + 16 * nr - 1) / (16 * nr), many = 256 / (tiles * z);
    const dim3 grid((unsigned)tiles, (unsigned)(many < 1 ? 1 : many > LORA_TOKENS ? LORA_TOKENS : many), (unsigned)z);
    const dim3 block(64 * lora_waves(nr));
    if (nr == 1) hipLaunchKernelGGL((lora_down_kernel<1>), grid, block, 0, s, a);
    else if (nr == 2) hipLaunchKernelGGL((lora_down_kernel<2>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((lora_down_kernel<4>), grid, block, 0, s, a);
    return (int)hipGetLastError();
}

int64_t lora_up_groups(int64_t M, int64_t N) {
    const int64_t tokens = LORA_TOKENS * LORA_UP_WAVES;
    return ((M + tokens - 1) / tokens) * ((N + LORA_COLS - 1) / LORA_COLS);
}

template <bool YF, bool OF>
static int launch_up(const LoraArgs& a, hipStream_t s) {
    if (a.M <= LORA_FEW) {
        auto launch = [&](auto lanes) {
            constexpr int G = decltype(lanes)::value, C = 4 * lora_few_loads(G) * (64 / G);
            hipLaunchKernelGGL((lora_up_few_kernel<YF, OF, G>), dim3((unsigned)((a.N + C - 1) / C), (unsigned)a.M), dim3(256), 0, s, a);
        };
        if (a.r <= 8) launch(std::integral_constant<int, 1>{});
        else if (a.r <= 16) launch(std::integral_constant<int, 2>{});
        else if (a.r <= 32) launch(std::integral_constant<int, 4>{});
        else if (a.r <= 64) launch(std::integral_constant<int, 8>{});
        else if (a.r <= 128) launch(std::integral_constant<int, 16>{});
        else launch(std::integral_constant<int, 32>{});
        return (int)hipGetLastError();
    }
    const int64_t cols = (a.N + LORA_COLS - 1) / LORA_COLS, tiles = lora_up_groups(a.M, LORA_COLS);
    // as many columns a workgroup as leave two of them for each CU (one where its registers have room for no more):
    // all run at once, and a workgroup's way in is spread over its columns.  4096 tokens x 4096, rank 64, us:
    // 4096 workgroups of 64 columns 37, 2048 29, 1024 25, 512 23, 256 32.
    const int64_t room = a.r > 128 ? 256 : 512;
    int64_t chunks = (tiles * cols + room - 1) / room;
    if (chunks > cols) chunks = cols;
    const dim3 grid((unsigned)(tiles * ((cols + chunks - 1) / chunks))), block(64 * LORA_UP_WAVES);
    auto launch = [&](auto whole_c) {
        constexpr bool WHOLE = decltype(whole_c)::value;
        if (a.r <= 32) hipLaunchKernelGGL((lora_up_kernel<YF, OF, 1, WHOLE>), grid, block, 0, s, a, (int)chunks);
        else if (a.r <= 64) hipLaunchKernelGGL((lora_up_kernel<YF, OF, 2, WHOLE>), grid, block, 0, s, a, (int)chunks);
        else if (a.r <= 128) hipLaunchKernelGGL((lora_up_kernel<YF, OF, 4, WHOLE>), grid, block, 0, s, a, (int)chunks);
        else hipLaunchKernelGGL((lora_up_kernel<YF, OF, 8, WHOLE>), grid, block, 0, s, a, (int)chunks);
    };
    if (a.N % LORA_COLS == 0) launch(std::true_type{});
    else launch(std::false_type{});
    return (int)hipGetLastError();
}

int launch_lora_up(const LoraArgs& a, int y_f32, int out_f32, hipStream_t s) {
    return !y_f32 ? launch_up<false, false>(a, s) : out_f32 ? launch_up<true, true>(a, s) : launch_up<true, false>(a, s);
}

int launch_lora_add(int f32, int64_t M, int64_t N, int64_t K, int64_t r, int64_t L, const void* x, int64_t ldx,
                    const int32_t* adapters, const void* lora_a, const void* lora_b, const float* scales, const void* y,
                    int64_t ldy, void* out, int64_t ldo, float* workspace, void* hip_stream) {
    if (M == 0 || N == 0) return 0;
    hipStream_t s = (hipStream_t)hip_stream;
    const LoraArgs a{M, N, K, (int)r, L, (const uint16_t*)x, ldx, adapters, (const uint16_t*)lora_a, (const uint16_t*)lora_b,
                     scales, workspace, y, ldy, out, ldo};
    const int e = M <= LORA_FEW ? launch_lora_down_few(a, s) : launch_lora_down_many(a, s);
    return e ? e : launch_lora_up(a, f32, f32, s);
}

}  // namespace bsq
