// embedding.hip -- scaled rows of the int8 embedding matrix, and the embedding's gradient (gfx950).
//
//   lookup:    out[t] = (scale s_e[id]) e[id],  id = tokens[t]         (zeros outside [0, V))
//   backward:  de[v] (+)= scale sum over the t with tokens[t] = v of dout[t]
//
// The gradient is a scatter of T rows into V, with rows hit any number of times.  Float atomics
// would add in an order that changes from run to run, so the tokens are sorted (up to 8192 by counting, more in
// stable radix passes of 8 bits; equal tokens stay in their order) and each row's sum runs over its tokens in order.  The sorted list
// is cut into pieces of equal length, so that a token that fills half the batch is summed by many
// workgroups: a piece writes the rows that lie wholly in it, and the sums of a row that crosses its
// ends go to the workspace, from where a second kernel joins them in order.
#include "device_common.h"

namespace dfssm {

namespace {

// ---------------------------------------------------------------- lookup
constexpr int kLookTokens = 4;  // tokens per thread: independent loads in flight

template <bool kBf16, int VEC>
__global__ __launch_bounds__(256) void lookup_scaled_kernel(const int32_t* __restrict__ tokens, int64_t T,
                                                            const int8_t* __restrict__ e,
                                                            const float* __restrict__ s_e, int64_t V, int64_t K,
                                                            float scale, void* __restrict__ out, int64_t ldo) {
    int64_t k = ((int64_t)blockIdx.y * 256 + threadIdx.x) * VEC;
    if (k >= K) return;
    k = k + VEC <= K ? k : K - VEC;  // (a row's last vector may overlap the one before: both write the same)
    const int64_t t0 = (int64_t)blockIdx.x * kLookTokens;
    int64_t id[kLookTokens];
    float s[kLookTokens];
    int8_t c[kLookTokens][VEC];
#pragma unroll
    for (int j = 0; j < kLookTokens; ++j) id[j] = tokens[t0 + j < T ? t0 + j : T - 1];
#pragma unroll
    for (int j = 0; j < kLookTokens; ++j) {
        const bool in = id[j] >= 0 && id[j] < V;
        const int64_t row = in ? id[j] : 0;
        s[j] = in ? scale * s_e[row] : 0.0f;
        __builtin_memcpy(c[j], e + row * K + k, VEC);
        if (!in)
#pragma unroll
            for (int i = 0; i < VEC; ++i) c[j][i] = 0;
    }
#pragma unroll
    for (int j = 0; j < kLookTokens; ++j) {
        if (t0 + j >= T) break;
        const int64_t at = (t0 + j) * ldo + k;
        if constexpr (kBf16) {
            uint16_t o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = (uint16_t)bf16_bits(s[j] * (float)c[j][i]);
            __builtin_memcpy(static_cast<uint16_t*>(out) + at, o, VEC * 2);
        } else {
            float o[VEC];
#pragma unroll
            for (int i = 0; i < VEC; ++i) o[i] = s[j] * (float)c[j][i];
            __builtin_memcpy(static_cast<float*>(out) + at, o, VEC * 4);
        }
    }
}

// ---------------------------------------------------------------- sort
// A workgroup of W waves sorts blocks of W * R * 64 items: wave w owns R rounds of 64 in a row, so
// (wave, round, lane) is the items' order.

// Lanes of the wave whose digit equals this lane's (dead lanes share digit 256).
__device__ __forceinline__ uint64_t same_digit(int digit) {
    uint64_t m = ~0ull;
#pragma unroll
    for (int b = 0; b < 9; ++b) {
        const uint64_t set = __ballot((digit >> b) & 1);
        m &= (digit >> b) & 1 ? set : ~set;
    }
    return m;
}

template <int W>
struct SortShared {
    int32_t count[W][256];  // per wave and digit; then the wave's first rank within the block
    int32_t total[256];     // the block's items of a digit
    int32_t start[256];     // where the block's items of a digit go
};

// Ranks of a block's items by digit: rank[r] counts the block's earlier items with the same digit.
// sh.total is complete after the call (a barrier ends it).
template <int W, int R>
__device__ __forceinline__ void block_ranks(const uint32_t (&key)[R], const bool (&live)[R], int shift,
                                            SortShared<W>& sh, int (&digit)[R], int (&rank)[R]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    for (int d = lane; d < 256; d += 64) sh.count[wave][d] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
        digit[r] = live[r] ? (int)((key[r] >> shift) & 255u) : 256;
        const uint64_t same = same_digit(digit[r]);
        const int before = __popcll(same & ((1ull << lane) - 1));
        rank[r] = 0;
        if (live[r]) rank[r] = sh.count[wave][digit[r]] + before;
        wave_lds_order();  // every lane's read comes before the adds, and they before the next round's reads
        if (live[r] && before == 0) sh.count[wave][digit[r]] += __popcll(same);
        wave_lds_order();
    }
    __syncthreads();
    if (threadIdx.x < 256) {
        int sum = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const int c = sh.count[w][threadIdx.x];
            sh.count[w][threadIdx.x] = sum;
            sum += c;
        }
        sh.total[threadIdx.x] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (live[r]) rank[r] += sh.count[wave][digit[r]];
}

// Exclusive scan of 256 values, one per thread of the first four waves; all threads call it.
__device__ __forceinline__ int scan256(int v, int32_t* part) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(inc, d);
        if (lane >= d) inc += o;
    }
    if (lane == 63 && wave < 4) part[wave] = inc;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < wave && w < 4; ++w) base += part[w];
    __syncthreads();
    return base + inc - v;
}

// A token's sort key: tokens outside the vocabulary sort behind all others.
__device__ __forceinline__ uint32_t token_key(int32_t id, uint32_t V) { return id >= 0 && (uint32_t)id < V ? (uint32_t)id : V; }

// Few tokens: a token's place is the number of tokens with a smaller key and of earlier ones with the same.
// A group places 64 tokens, one a lane; its 16 waves share the keys, which are uniform and come as scalar loads,
// two vector instructions a key (4096 tokens 9.9 us; radix passes by one workgroup took 12.8).  The key is the id as an
// unsigned number: ids outside the vocabulary come behind all others, in any order.
constexpr int kRankMost = 8192, kRankWaves = 16;

__global__ __launch_bounds__(kRankWaves * 64) void sort_rank_kernel(const uint32_t* __restrict__ tokens, int T,
                                                                    uint32_t* __restrict__ keys,
                                                                    int32_t* __restrict__ order) {
    __shared__ int32_t part[kRankWaves][64];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
    const int b0 = (int)blockIdx.x * 64, b1 = b0 + 64 < T ? b0 + 64 : T, t = b0 + lane;
    const uint32_t key = tokens[t < T ? t : T - 1];
    // (a multiple of 64: the group's own tokens are one wave's, and loads are aligned)
    const int share = (T + kRankWaves * 64 - 1) / (kRankWaves * 64) * 64;
    const int begin = wave * share, end = begin + share < T ? begin + share : T;
    int place = 0;
    // earlier tokens count where their key is the same, too
    const int e0 = end < b0 ? end : b0;
#pragma unroll 32
    for (int j = begin; j < e0; ++j) place += tokens[j] <= key;
    if (begin <= b0 && b0 < end) {  // the group's own tokens: the lanes hold them
#pragma unroll
        for (int i = 0; i < 64; ++i) {
            const uint32_t k = (uint32_t)__builtin_amdgcn_readlane((int)key, i);
            if (i < b1 - b0) place += i < lane ? k <= key : k < key;
        }
    }
#pragma unroll 32
    for (int j = begin > b1 ? begin : b1; j < end; ++j) place += tokens[j] < key;
    part[wave][lane] = place;
    __syncthreads();
    if (wave == 0 && t < T) {
        int at = 0;
#pragma unroll
        for (int w = 0; w < kRankWaves; ++w) at += part[w][lane];
        keys[at] = key;
        order[at] = t;
    }
}

// Many tokens, blocks of 512 R items.  A pass is two kernels: how often each digit occurs in each block ...
// (`tokens` on the first pass, (keys, order) afterwards.  Counting for the next pass inside the scatter saves a
// launch, but a token that fills much of the batch sends that many atomics to one count: 15.7 us against 5 + 4.6.)
constexpr int kManyWaves = 8, kManyThreads = kManyWaves * 64;

__global__ __launch_bounds__(kManyThreads) void sort_count_kernel(const int32_t* __restrict__ tokens,
                                                                  const uint32_t* __restrict__ keys, int64_t T,
                                                                  uint32_t V, int block, int shift,
                                                                  int32_t* __restrict__ hist) {
    __shared__ int32_t count[256];
    if (threadIdx.x < 256) count[threadIdx.x] = 0;
    __syncthreads();
    const int64_t b0 = (int64_t)blockIdx.x * block;
    for (int r = 0; r < block; r += kManyThreads) {
        const int64_t i = b0 + r + threadIdx.x;
        if (i < T) atomicAdd(&count[((keys ? keys[i] : token_key(tokens[i], V)) >> shift) & 255u], 1);
    }
    __syncthreads();
    if (threadIdx.x < 256) hist[(int64_t)blockIdx.x * 256 + threadIdx.x] = count[threadIdx.x];
}

// ... and the block's items to their places, behind all smaller digits and the digit's items of the blocks before.
template <int R>
__global__ __launch_bounds__(kManyThreads) void sort_scatter_kernel(const int32_t* __restrict__ tokens,
                                                                    const uint32_t* __restrict__ keys,
                                                                    const int32_t* __restrict__ order, int64_t T,
                                                                    uint32_t V, int shift,
                                                                    const int32_t* __restrict__ hist,
                                                                    uint32_t* __restrict__ keys_out,
                                                                    int32_t* __restrict__ order_out) {
    constexpr int kBlock = kManyThreads * R;
    __shared__ SortShared<kManyWaves> sh;
    __shared__ int32_t part[4];
    __shared__ int32_t halves[2][256][2];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t key[R];
    int32_t idx[R];
    bool live[R];
    int digit[R], rank[R];
    const int64_t i0 = (int64_t)blockIdx.x * kBlock + wave * R * 64 + lane;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int64_t i = i0 + r * 64;
        live[r] = i < T;
        idx[r] = live[r] ? (order ? order[i] : (int32_t)i) : 0;
        key[r] = live[r] ? (keys ? keys[i] : token_key(tokens[i], V)) : 0u;
    }
    // digit d's count in the blocks before this one and in all (two halves of the threads share the blocks)
    const int d = threadIdx.x & 255;
    {
        const int h = threadIdx.x >> 8, n = (int)gridDim.x;
        int before = 0, all = 0;
        for (int b0 = h; b0 < n; b0 += 16) {
            int c[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = b0 + 2 * j < n ? hist[(int64_t)(b0 + 2 * j) * 256 + d] : 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                all += c[j];
                before += b0 + 2 * j < (int)blockIdx.x ? c[j] : 0;
            }
        }
        halves[h][d][0] = before;
        halves[h][d][1] = all;
    }
    __syncthreads();
    const int total = halves[0][d][1] + halves[1][d][1];
    const int start = scan256(threadIdx.x < 256 ? total : 0, part);
    if (threadIdx.x < 256) sh.start[d] = start + halves[0][d][0] + halves[1][d][0];
    block_ranks<kManyWaves, R>(key, live, shift, sh, digit, rank);
#pragma unroll
    for (int r = 0; r < R; ++r)
        if (live[r]) {
            const int at = sh.start[digit[r]] + rank[r];
            keys_out[at] = key[r];
            order_out[at] = idx[r];
        }
}

// ---------------------------------------------------------------- sums
struct SumArgs {
    const uint32_t* keys;   // sorted
    const int32_t* order;
    int64_t T;
    const void* dout;
    int64_t ldd;
    uint32_t V;
    int64_t K;
    float scale;
    void* de;
    float* head;            // [pieces][K]: a piece's part of the row that began before it
    float* tail;            // [pieces][K]: its part of a row that begins in it and goes on behind it
    int64_t piece;          // sorted tokens per piece
    int pieces, col_blocks;
    int fill_rows;          // per workgroup that writes zeros: 8 or kFillRows
};

template <bool kBf16, int VEC>
__device__ __forceinline__ void load_vec(const void* base, int64_t at, float (&v)[VEC]) {
    if constexpr (kBf16) {
        uint16_t b[VEC];
        __builtin_memcpy(b, static_cast<const uint16_t*>(base) + at, VEC * 2);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[i] = __uint_as_float((uint32_t)b[i] << 16);
    } else {
        __builtin_memcpy(v, static_cast<const float*>(base) + at, VEC * 4);
    }
}

template <bool kBf16, int VEC>
__device__ __forceinline__ void store_vec(void* base, int64_t at, const float (&v)[VEC]) {
    if constexpr (kBf16) {
        uint16_t b[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) b[i] = (uint16_t)bf16_bits(v[i]);
        __builtin_memcpy(static_cast<uint16_t*>(base) + at, b, VEC * 2);
    } else {
        __builtin_memcpy(static_cast<float*>(base) + at, v, VEC * 4);
    }
}

// Zeros; past the caches where de is larger than they are (412 MB: the sums and zeros of 16384 tokens 89 against
// 93 us, and the parts of crossing rows stay cached: their join 7.4 against 9.3).
template <bool kBf16, int VEC, bool kStream>
__device__ __forceinline__ void store_zeros(void* base, int64_t at) {
    if constexpr (kStream) {
        static_assert(VEC == 4, "streamed in vectors");
        typedef uint32_t v2u __attribute__((ext_vector_type(2)));
        if constexpr (kBf16) __builtin_nontemporal_store((v2u){0, 0}, reinterpret_cast<v2u*>(static_cast<uint16_t*>(base) + at));
        else __builtin_nontemporal_store((v4f){0, 0, 0, 0}, reinterpret_cast<v4f*>(static_cast<float*>(base) + at));
    } else {
        const float zero[VEC] = {};
        store_vec<kBf16, VEC>(base, at, zero);
    }
}

// skip: elements of the vector that the thread before writes.
template <bool kOutBf16, bool kAdd, int VEC>
__device__ __forceinline__ void write_row(const SumArgs& a, uint32_t row, int64_t k, int skip, const float (&sum)[VEC]) {
    float o[VEC];
    const int64_t at = (int64_t)row * a.K + k;
    if constexpr (kAdd) {
        load_vec<kOutBf16, VEC>(a.de, at, o);
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] += a.scale * sum[i];
        if (skip) {  // (added once)
#pragma unroll
            for (int i = 1; i < VEC; ++i) {
                const float one[1] = {o[i]};
                if (i >= skip) store_vec<kOutBf16, 1>(a.de, at + i, one);
            }
            return;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) o[i] = a.scale * sum[i];
    }
    store_vec<kOutBf16, VEC>(a.de, at, o);
}

// A row's vectors may start anywhere in memory; its last one is moved back to end with the row and overlaps the one
// before by the returned number of elements, which both compute alike (16384 tokens of width 2049 125 us, element by
// element 161; width 2048 114).
template <int VEC>
__device__ __forceinline__ int row_vector(int64_t& k, int64_t K) {
    const int64_t over = k + VEC - K;
    if (over <= 0) return 0;
    k -= over;
    return (int)over;
}

constexpr int kFillRows = 32;  // rows at most per workgroup that fills the rows without tokens

// Workgroups [0, pieces * col_blocks) sum pieces; the ones behind them (none when adding to de) write zeros
// to the rows that no token names.
template <bool kInBf16, bool kOutBf16, bool kAdd, int VEC, bool kStream>
__global__ __launch_bounds__(256) void piece_sum_kernel(SumArgs a) {
    const int nsum = a.pieces * a.col_blocks;
    if ((int)blockIdx.x >= nsum) {
        if constexpr (!kAdd) {
            static_assert(kFillRows * 8 == 256, "8 lanes search a row");
            __shared__ int32_t named[kFillRows];
            const int64_t r0 = (int64_t)((int)blockIdx.x - nsum) * a.fill_rows;
            const int rows = (int)(a.V - r0 < a.fill_rows ? a.V - r0 : a.fill_rows);
            if (threadIdx.x < (unsigned)a.fill_rows * 8) {  // (whole waves: 8 rows each)
                // the first sorted token >= row, 8 probes a step
                const int j = threadIdx.x & 7, group = threadIdx.x & 56;
                const uint32_t row = (uint32_t)(r0 + (threadIdx.x >> 3));
                int lo = 0, hi = (int)a.T;
                while (__any(lo < hi)) {
                    const int len = hi - lo, p = lo + (int)((int64_t)len * (j + 1) / 9);
                    const bool less = len > 0 && a.keys[p] < row;
                    const int n = __popcll((__ballot(less) >> group) & 255);  // the probes below the row: the first n
                    const int below = lo + (int)((int64_t)len * n / 9), above = lo + (int)((int64_t)len * (n + 1) / 9);
                    if (len > 0) {
                        if (n < 8) hi = above;
                        if (n > 0) lo = below + 1;
                    }
                }
                if (j == 0) named[threadIdx.x >> 3] = lo < a.T && a.keys[lo] == row;
            }
            __syncthreads();
            if (a.K % VEC == 0 && a.K >= 256 * VEC) {
                for (int r = 0; r < rows; ++r)
                    if (!named[r])
                        for (int64_t k = threadIdx.x * VEC; k < a.K; k += 256 * VEC)
                            store_zeros<kOutBf16, VEC, kStream>(a.de, (r0 + r) * a.K + k);
            } else {
                // the group's rows as one run of vectors, which rows need not start with: rows of odd width still take
                // whole aligned lines, and narrow rows all the threads
                const uint32_t K = (uint32_t)a.K, n = (uint32_t)rows * K;
                const float per = 1.0f / (float)K;
#pragma unroll 4
                for (uint32_t i = threadIdx.x * VEC; i < n; i += 256 * VEC) {
                    uint32_t r = (uint32_t)((float)i * per);  // (i < 2^22: off by one at the most)
                    r = r * K > i ? r - 1 : (r + 1) * K <= i ? r + 1 : r;
                    const uint32_t next = (r + 1) * K;        // K >= VEC: the vector reaches at most one row more
                    if (i + VEC <= n && !named[r] && (i + VEC <= next || !named[r + 1])) {
                        store_zeros<kOutBf16, VEC, kStream>(a.de, r0 * a.K + i);
                    } else {
#pragma unroll
                        for (int j = 0; j < VEC; ++j)
                            if (i + j < n && !named[i + j < next ? r : r + 1])
                                store_zeros<kOutBf16, 1, false>(a.de, r0 * a.K + i + j);
                    }
                }
            }
        }
        return;
    }
    const int piece = (int)blockIdx.x / a.col_blocks, cb = (int)blockIdx.x - piece * a.col_blocks;
    int64_t k = ((int64_t)cb * 256 + threadIdx.x) * VEC;
    const int64_t p0 = piece * a.piece, p1 = p0 + a.piece < a.T ? p0 + a.piece : a.T;
    if (k >= a.K) return;
    const int skip = row_vector<VEC>(k, a.K);
    const bool from_before = p0 > 0 && a.keys[p0 - 1] == a.keys[p0];
    const bool goes_on = p1 < a.T && a.keys[p1] == a.keys[p1 - 1];
    float sum[VEC] = {};
    bool first = true;  // still in the piece's first row
    constexpr int U = 8;  // rows in flight
    for (int64_t p = p0; p < p1; p += U) {
        float v[U][VEC];
        uint32_t key[U + 1];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t q = p + j < p1 ? p + j : p1 - 1;
            key[j] = a.keys[q];
            load_vec<kInBf16, VEC>(a.dout, a.order[q] * a.ldd + k, v[j]);
        }
        key[U] = p + U < p1 ? a.keys[p + U] : 0xffffffffu;
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (p + j >= p1) break;
#pragma unroll
            for (int i = 0; i < VEC; ++i) sum[i] += v[j][i];
            const bool last = p + j + 1 == p1;
            if (last || key[j + 1] != key[j]) {
                if (key[j] < a.V) {
                    if (first && from_before) store_vec<false, VEC>(a.head, piece * a.K + k, sum);
                    else if (last && goes_on) store_vec<false, VEC>(a.tail, piece * a.K + k, sum);
                    else write_row<kOutBf16, kAdd, VEC>(a, key[j], k, skip, sum);
                }
                first = false;
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum[i] = 0.0f;
            }
        }
    }
}

// Rows that cross pieces: the piece where a row begins adds the following pieces' parts in order.
template <bool kOutBf16, bool kAdd, int VEC>
__global__ __launch_bounds__(256) void piece_join_kernel(SumArgs a) {
    const int piece = (int)blockIdx.x / a.col_blocks, cb = (int)blockIdx.x - piece * a.col_blocks;
    int64_t k = ((int64_t)cb * 256 + threadIdx.x) * VEC;
    const int64_t p0 = piece * a.piece, p1 = p0 + a.piece;
    if (k >= a.K || p1 >= a.T) return;
    const int skip = row_vector<VEC>(k, a.K);
    const uint32_t row = a.keys[p1 - 1];
    if (row >= a.V || a.keys[p1] != row) return;                    // nothing goes on
    if (p0 > 0 && a.keys[p0] == row && a.keys[p0 - 1] == row) return;  // it began before this piece
    float sum[VEC];
    load_vec<false, VEC>(a.tail, piece * a.K + k, sum);
    constexpr int U = 8;  // parts in flight
    for (int q = piece + 1; q < a.pieces; q += U) {
        uint32_t key[U];
        float v[U][VEC];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t p = q + j < a.pieces ? q + j : a.pieces - 1;
            key[j] = a.keys[p * a.piece];
            load_vec<false, VEC>(a.head, p * a.K + k, v[j]);  // (may be no part of the row: not added then)
        }
        int n = 0;  // parts of the row: the first ones, since the keys are sorted
#pragma unroll
        for (int j = 0; j < U; ++j) n += q + j < a.pieces && key[j] == row ? 1 : 0;
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (j < n)
#pragma unroll
                for (int i = 0; i < VEC; ++i) sum[i] += v[j][i];
        if (n < U) break;
    }
    write_row<kOutBf16, kAdd, VEC>(a, row, k, skip, sum);
}

// How a backward call's workspace lies.
struct Plan {
    int64_t piece;
    int pieces, sort_block, sort_blocks, passes;
    size_t keys[2], order[2], hist, head, tail, bytes;
};

Plan make_plan(int64_t T, int64_t V, int64_t K) {
    Plan p{};
    // pieces of 8 tokens (one batch of loads: 4096 tokens of width 2048 20.3 us against 30.5 in pieces of 32), longer ones
    // past 8192 tokens, where 1024 pieces fill the GPU and shorter ones only leave more to join (16384 tokens: 104
    // against 96 us)
    p.piece = T <= kRankMost ? 8 : ((T + 1023) / 1024 + 31) / 32 * 32;
    p.pieces = (int)((T + p.piece - 1) / p.piece);
    // radix passes in blocks of 1024 tokens; of 4096 where so many blocks' counts would take long to add up
    // (each block reads all: 2^22 tokens of width 64 1.0 ms in all, 2^24 of width 16 5.6)
    p.sort_block = T <= 65536 ? kManyThreads * 2 : kManyThreads * 8;
    p.sort_blocks = T <= kRankMost ? 0 : (int)((T + p.sort_block - 1) / p.sort_block);
    p.passes = 1;
    while (p.passes < 4 && ((uint64_t)V >> (8 * p.passes)) != 0) ++p.passes;  // keys 0 .. V
    size_t at = 0;
    auto take = [&](int64_t b) {
        const size_t was = at;
        at += ((size_t)b + 255) / 256 * 256;
        return was;
    };
    for (int i = 0; i < 2; ++i) {
        p.keys[i] = take(T * 4);
        p.order[i] = take(T * 4);
    }
    // Room that no shorter batch's plan needs more of: its pieces, 8 tokens each up to 1024 of them, and its blocks, at
    // most 64 up to 65536 tokens.
    const int64_t rows = T < kRankMost ? (T + 7) / 8 : 1024;
    p.hist = take((int64_t)(T > 65536 && p.sort_blocks < 64 ? 64 : p.sort_blocks) * 256 * 4);
    p.head = take(rows * K * 4);
    p.tail = take(rows * K * 4);
    p.bytes = at;
    return p;
}

template <bool kInBf16, bool kOutBf16, bool kAdd, int VEC>
hipError_t launch_sums(SumArgs a, hipStream_t stream) {
    a.col_blocks = (int)((a.K + 256 * VEC - 1) / (256 * VEC));
    // (8 where 32 would leave the GPU unfilled: 200 tokens x 1500 rows of width 3000 13 us against 19)
    a.fill_rows = a.V >= 32768 ? kFillRows : 8;
    const int64_t fills = kAdd ? 0 : ((int64_t)a.V + a.fill_rows - 1) / a.fill_rows;
    const dim3 grid((unsigned)((int64_t)a.pieces * a.col_blocks + fills));
    constexpr bool kMayStream = !kAdd && VEC == 4;
    if (kMayStream && ((uintptr_t)a.de & 15u) == 0 && (int64_t)a.V * a.K * (kOutBf16 ? 2 : 4) > (int64_t)160 << 20)
        piece_sum_kernel<kInBf16, kOutBf16, kAdd, VEC, kMayStream><<<grid, 256, 0, stream>>>(a);
    else
        piece_sum_kernel<kInBf16, kOutBf16, kAdd, VEC, false><<<grid, 256, 0, stream>>>(a);
    if (hipError_t err = hipGetLastError()) return err;
    if (a.pieces > 1)
        piece_join_kernel<kOutBf16, kAdd, VEC><<<dim3((unsigned)(a.pieces * a.col_blocks)), 256, 0, stream>>>(a);
    return hipGetLastError();
}

template <bool kInBf16, bool kOutBf16>
hipError_t launch_sums_t(const SumArgs& a, bool add, bool vec, hipStream_t stream) {
    if (add) return vec ? launch_sums<kInBf16, kOutBf16, true, 4>(a, stream) : launch_sums<kInBf16, kOutBf16, true, 1>(a, stream);
    return vec ? launch_sums<kInBf16, kOutBf16, false, 4>(a, stream) : launch_sums<kInBf16, kOutBf16, false, 1>(a, stream);
}

template <bool kBf16>
hipError_t launch_lookup_t(const int32_t* tokens, int64_t T, const int8_t* e, const float* s_e, int64_t V, int64_t K,
                           float scale, void* out, int64_t ldo, hipStream_t stream) {
    constexpr int VEC = kBf16 ? 8 : 4;  // 16 bytes of output a thread
    const bool vec = K >= VEC;
    const int64_t per = 256 * (vec ? VEC : 1);
    constexpr int64_t kSlice = (int64_t)1 << 24;  // tokens per launch: its threads stay below 2^32
    for (int64_t t0 = 0; t0 < T; t0 += kSlice) {
        const int64_t n = T - t0 < kSlice ? T - t0 : kSlice;
        void* const o = static_cast<uint8_t*>(out) + t0 * ldo * (kBf16 ? 2 : 4);
        const dim3 grid((unsigned)((n + kLookTokens - 1) / kLookTokens), (unsigned)((K + per - 1) / per));
        if (vec) lookup_scaled_kernel<kBf16, VEC><<<grid, 256, 0, stream>>>(tokens + t0, n, e, s_e, V, K, scale, o, ldo);
        else lookup_scaled_kernel<kBf16, 1><<<grid, 256, 0, stream>>>(tokens + t0, n, e, s_e, V, K, scale, o, ldo);
        if (hipError_t err = hipGetLastError()) return err;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_embedding_lookup_scaled(const int32_t* tokens, int64_t T, const int8_t* e, const float* s_e,
                                          int64_t V, int64_t K, float scale, void* out, int64_t ldo, bool bf16,
                                          hipStream_t stream) {
    return bf16 ? launch_lookup_t<true>(tokens, T, e, s_e, V, K, scale, out, ldo, stream)
                : launch_lookup_t<false>(tokens, T, e, s_e, V, K, scale, out, ldo, stream);
}

size_t embedding_backward_workspace_bytes(int64_t T, int64_t V, int64_t K) { return make_plan(T, V, K).bytes; }

hipError_t launch_embedding_backward(const int32_t* tokens, int64_t T, const void* dout, int64_t ldd, bool dout_bf16,
                                     int64_t V, int64_t K, float scale, void* de, bool de_bf16, bool accumulate,
                                     void* workspace, hipStream_t stream) {
    const Plan p = make_plan(T, V, K);
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    uint32_t* keys[2] = {reinterpret_cast<uint32_t*>(ws + p.keys[0]), reinterpret_cast<uint32_t*>(ws + p.keys[1])};
    int32_t* order[2] = {reinterpret_cast<int32_t*>(ws + p.order[0]), reinterpret_cast<int32_t*>(ws + p.order[1])};
    int32_t* hist = reinterpret_cast<int32_t*>(ws + p.hist);
    int at = 0;
    if (p.sort_blocks == 0) {
        sort_rank_kernel<<<dim3((unsigned)((T + 63) / 64)), kRankWaves * 64, 0, stream>>>(
            reinterpret_cast<const uint32_t*>(tokens), (int)T, keys[0], order[0]);
    } else {
        const dim3 grid((unsigned)p.sort_blocks);
        for (int i = 0; i < p.passes; ++i) {
            const uint32_t* kin = i ? keys[at] : nullptr;
            const int32_t* oin = i ? order[at] : nullptr;
            const int to = i ? at ^ 1 : 0;
            sort_count_kernel<<<grid, kManyThreads, 0, stream>>>(tokens, kin, T, (uint32_t)V, p.sort_block, 8 * i, hist);
            if (p.sort_block == kManyThreads * 2)
                sort_scatter_kernel<2><<<grid, kManyThreads, 0, stream>>>(tokens, kin, oin, T, (uint32_t)V, 8 * i, hist, keys[to], order[to]);
            else
                sort_scatter_kernel<8><<<grid, kManyThreads, 0, stream>>>(tokens, kin, oin, T, (uint32_t)V, 8 * i, hist, keys[to], order[to]);
            at = to;
        }
    }
    if (hipError_t err = hipGetLastError()) return err;
    const SumArgs a{keys[at], order[at], T, dout, ldd, (uint32_t)V, K, scale, de,
                    reinterpret_cast<float*>(ws + p.head), reinterpret_cast<float*>(ws + p.tail), p.piece, p.pieces, 0, 0};
    const bool vec = K >= 4;
    if (dout_bf16) return de_bf16 ? launch_sums_t<true, true>(a, accumulate, vec, stream) : launch_sums_t<true, false>(a, accumulate, vec, stream);
    return de_bf16 ? launch_sums_t<false, true>(a, accumulate, vec, stream) : launch_sums_t<false, false>(a, accumulate, vec, stream);
}

}  // namespace dfssm
