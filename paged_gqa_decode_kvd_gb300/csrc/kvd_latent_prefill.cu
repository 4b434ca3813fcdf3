// kvd_latent_prefill.cu — expanded latent attention: every head has its own 128 dims of key and of value, the 64
// rotated dims of the key are one vector a token.
//
// Row (token i of the T rows of request b, head h) over its N keys, causal: t ≤ N − T + i:
//   l_t = scale·(<q[:128], k_t,h> + <q[128:], r_t>),  out = Σ_t softmax(l)_t·v_t,h,  lse = log Σ exp(l_t).
//
// One CTA per SM takes units of 256 tokens of one head: two softmax warpgroups of 128 rows, a thread a row, that share every tile of 128
// keys.  A producer warp copies Q (96 KiB) and, through one ring of eight 16 KiB pieces, a tile's K (twice 64 dims, then the rotated ones,
// which all heads share) and V (twice 64 keys) by TMA; V is read N-major, as it lands.  An issuing warp for each warpgroup: S = Q·Kᵀ from
// shared memory, P over S in tensor memory, O += P·V.  A piece is free when both have used it.  The reference maximum moves only when a row's
// passes it by 8.
// Rounding: q, k, v enter exactly, logits, statistics and sums are fp32.  Where out is bf16 a weight enters as one bf16 (off by at most 2^-8
// of itself; its sum is taken before): outputs are 1.2 to 1.4 times as far from 64 bits as an fp32 form's rounded to bf16; divided by the sum of
// the weights as they were rounded (as in the absorbed kernel) they are no nearer, and the call takes 11% longer.  Where out is fp32 (TWO) nothing
// behind it hides that, so a weight enters as two bf16, cut off and its rest (off by at most 2^-15 of itself), for 40% more MMAs: 628 us
// in place of 454 for the prompt below.
//
// Bound: a whole prompt of 8,192, 32 heads: 453 us, 1,515 TFLOP/s (79% of measured; in a row of seconds, at the power cap and 1,920 MHz,
// 485 us, 83% of the rate measured so).  A tile takes both warpgroups 3,600 cycles, its MMAs 2,750 (S 12 x 71, at the limit of shared memory's 128 bytes a cycle, O 8 x 65 each), a softmax 1,300 beside the other's MMAs; the rest is what the
// turns leave between two runs.  Ragged prompts: 119 us against 53 of HBM: a unit's first tile waits 3 us for Q and K, its rows take 1 to 2 us,
// and rows of at most 128 tokens leave a warpgroup idle.
//
// Waits.  Each barrier's waiter is at most one phase behind it.  Every wait gives up after a second or so (200,000 tries; a barrier's suspends
// 3.8 us, a turn's sleeps as long once the first thousand have failed; not while a row is computed again, which ends by itself and takes
// 0.5 us a position); the kernel then reports it and ends.
#include <cuda.h>

#include "kvd_latent.h"
#include "kvd_tcgen.cuh"

namespace kvd {
namespace {

constexpr int kTile = 128;             // keys per tile
constexpr int kRows = 128;             // rows of a softmax warpgroup: one MMA
constexpr int kPieces = 8, kPieceBytes = 16384, kTilePieces = 5;   // K: three times 64 dims of 128 keys; V: twice 64 keys
constexpr int kChunk = kRows * 128;    // 64 dims of Q's rows
constexpr int kThreads = 384;
constexpr int kProducerWarp = 8, kIssueWarp = 9;   // the issuers are two
constexpr int kReaders = 10;           // warps that read a unit's description
constexpr float kLazy = 8.f;           // log2: how far a row's maximum may pass its reference
constexpr int kTries = 200000;         // tries of a wait, which suspend: a second or so
constexpr int kQuickTries = 1000;      // of a turn, which do not, before they sleep
constexpr uint32_t kTryNs = 3800;      // a barrier's try
constexpr uint64_t kWaitNs = 1000000000ull;   // of what must land before the block leaves
constexpr uint32_t kColS = 0, kColO = 256;    // tensor memory columns: S (and P over it) 2 × 128, O 2 × 128
constexpr uint32_t kColRest = 64;             // what P's rounding left, from S on

constexpr int kSorted = 512;           // blocks of tokens that are put in order
constexpr int kBlockBits = 20;

struct Unit {
    int b, h, s0, T, k0, N;
    int tok0;                          // first token
    int tiles[2];                      // of the warpgroups' rows (−1: no rows)
    int end;                           // keys that the last row attends
    uint32_t turn[2];                  // of Q of each warpgroup
};

struct Smem {
    uint8_t q[2][3 * kChunk];
    uint8_t piece[kPieces][kPieceBytes];
    Unit unit[2];
    uint64_t full[kPieces], empty[kPieces], q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], u_full[2], u_empty[2], drain[2];
    uint32_t tmem;
    int turn;                          // the tensor cores are one issuer's
    int sorted;                        // blocks of 256 tokens in `order`, or −1
    uint32_t order[kSorted];           // request << 20 | block, dearest first
    volatile int abort;
    int again;                         // warps that compute a row again: every other wait may be longer for it
};

struct Maps {
    CUtensorMap q, k, v, r;
};

__device__ __forceinline__ bool wait_bar(Smem& s, uint64_t* bar, uint32_t phase) {
    #pragma unroll 1
    for (int i = 0; i < kTries; ++i) {
        if (__all_sync(kFull, mbar_try_wait(bar, phase & 1u))) return true;
        if (__any_sync(kFull, s.abort)) return false;
        if (i == kTries - 1 && __any_sync(kFull, *static_cast<volatile int*>(&s.again) > 0)) i = 0;
    }
    s.abort = 1;   // reported at the kernel's end
    return false;
}

// A barrier a lane (null: none), all of them with one vote.
__device__ __forceinline__ bool wait_lanes(Smem& s, uint64_t* bar, uint32_t phase) {
    #pragma unroll 1
    for (int i = 0; i < kTries; ++i) {
        if (__all_sync(kFull, !bar || mbar_try_wait(bar, phase & 1u))) return true;
        if (__any_sync(kFull, s.abort)) return false;
        if (i == kTries - 1 && __any_sync(kFull, *static_cast<volatile int*>(&s.again) > 0)) i = 0;
    }
    s.abort = 1;
    return false;
}

// Whether all of them are there already.
__device__ __forceinline__ bool test_lanes(uint64_t* bar, uint32_t phase) {
    uint32_t ok = 1;
    if (bar)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(smem_u32(bar)), "r"(phase & 1u)
            : "memory");
    return __all_sync(kFull, ok != 0);
}
// The tensor cores' queue is taken by one issuer at a time, for as long as it takes to issue a product's MMAs.  A try here does
// not suspend by itself: after the first ones, tens of microseconds of them, each is followed by a sleep, so that this wait's
// limit is the others' and its tries leave the softmax warps their issue slots.
__device__ __forceinline__ bool take_turn(Smem& s, int lane) {
    #pragma unroll 1
    for (int i = 0; i < kTries; ++i) {
        if (__any_sync(kFull, lane == 0 && atomicCAS(&s.turn, 0, 1) == 0)) return true;
        if (__any_sync(kFull, s.abort)) return false;
        if (i >= kQuickTries) __nanosleep(kTryNs);
        if (i == kTries - 1 && __any_sync(kFull, *static_cast<volatile int*>(&s.again) > 0)) i = 0;
    }
    s.abort = 1;
    return false;
}
__device__ __forceinline__ void give_turn(Smem& s, int lane) {
    __syncwarp();
    if (lane == 0) atomicExch(&s.turn, 0);
}

__device__ __forceinline__ void tma3(uint8_t* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.3d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void tma2(uint8_t* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
                 "l"(map), "r"(x), "r"(y), "r"(smem_u32(bar))
                 : "memory");
}

// ------------------------------------------------------------- one row, plainly
__device__ __forceinline__ void unpack4(float* x, const uint16_t* p) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    const float2 a = unpack_bf16(v.x), c = unpack_bf16(v.y);
    x[0] = a.x;
    x[1] = a.y;
    x[2] = c.x;
    x[3] = c.y;
}
// Whether a key of k0 + from .. k0 + to − 1 has a value that is not finite; by a warp.
__device__ __noinline__ bool odd_values(const LatentPrefillParams& p, int h, int64_t k0, int from, int to) {
    const int lane = threadIdx.x & 31;
    bool odd = false;
    #pragma unroll 1
    for (int64_t n = k0 + from; n < k0 + to; ++n) {
        float v[4];
        unpack4(v, p.v + n * p.v_stride + h * p.v_head + lane * 4);
        odd |= fmaf(v[0], 0.f, fmaf(v[1], 0.f, fmaf(v[2], 0.f, v[3] * 0.f))) != 0.f;   // (0·x is NaN unless x is finite)
    }
    return __any_sync(kFull, odd);
}
// A warp a row: a lane has four dims of k and v and two rotated ones.
__device__ __noinline__ void plain_row(const LatentPrefillParams& p, int64_t token, int h, int64_t k0, int end) {
    const int lane = threadIdx.x & 31;
    const int64_t row = token * p.n_q + h;
    float q[6], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, sum = 0.f;
    unpack4(q, p.q + row * kExpKey + lane * 4);
    const float2 qr = unpack_bf16(*reinterpret_cast<const uint32_t*>(p.q + row * kExpKey + kNope + lane * 2));
    q[4] = qr.x;
    q[5] = qr.y;
    for (int64_t n = k0; n < k0 + end; ++n) {
        float k[4], v[4];
        unpack4(k, p.k_nope + n * p.k_stride + h * p.k_head + lane * 4);
        unpack4(v, p.v + n * p.v_stride + h * p.v_head + lane * 4);
        const float2 rot = unpack_bf16(*reinterpret_cast<const uint32_t*>(p.k_rope + n * p.rope_stride + lane * 2));
        float dot = fmaf(q[4], rot.x, q[5] * rot.y);
        #pragma unroll
        for (int j = 0; j < 4; ++j) dot = fmaf(q[j], k[j], dot);
        #pragma unroll
        for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(kFull, dot, o);
        const float l = dot * p.scale_log2, top = fmaxf(m, l);
        const float ref = top == -INFINITY ? 0.f : top;
        const float f = exp2f(m - ref), w = exp2f(l - ref);
        m = top;
        sum = sum * f + w;
        #pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] = fmaf(w, v[j], acc[j] * f);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    #pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t at = row * kExpVal + lane * 4 + j;
        if (p.out_f32) static_cast<float*>(p.out)[at] = acc[j] * inv;
        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16(acc[j] * inv);
    }
    if (lane == 0 && p.lse_out) p.lse_out[row] = sum == 0.f ? -INFINITY : (m + log2f(sum)) * kLn2;
}

// ------------------------------------------------------------------ producer
// A unit is a block of 256 tokens of one head.  Blocks stand in order, the one with the most keys first (more than kSorted of
// them as they come: requests, within one its tokens from the last 256 on), and the heads of a block side by side.  CTA c of C
// takes the units c, 2C − 1 − c, 2C + c, 4C − 1 − c, ..: who has the dearer one of a turn has the cheaper of the next.
struct Span {
    int s0, T, k0, N;
    __device__ __forceinline__ int blocks() const { return (T + 2 * kRows - 1) / (2 * kRows); }
};
__device__ __forceinline__ Span load_span(const LatentPrefillParams& p, int b, bool tell) {
    Span x{p.q_start[b], 0, p.kv_start[b], 0};
    const int s1 = p.q_start[b + 1], k1 = p.kv_start[b + 1];
    if (x.s0 < 0 || s1 < x.s0 || s1 > p.n_tokens || x.k0 < 0 || k1 < x.k0 || k1 > p.n_keys) {
        if (tell) report(p.err, KVD_ERR_OOB);
        return x;
    }
    x.T = s1 - x.s0;
    x.N = k1 - x.k0;
    return x;
}
__device__ __forceinline__ int block_end(const LatentPrefillParams& p, const Span& x, int block) {   // keys its last row attends
    return p.causal ? max(0, x.N - x.T + min((block + 1) * 2 * kRows, x.T)) : x.N;
}
__device__ __forceinline__ void make_unit(const LatentPrefillParams& p, const Span& x, int b, int h, int block, Unit& u) {
    u.b = b;
    u.h = h;
    u.s0 = x.s0;
    u.T = x.T;
    u.k0 = x.k0;
    u.N = x.N;
    u.tok0 = block * 2 * kRows;
    u.end = 0;
    #pragma unroll
    for (int w = 0; w < 2; ++w) {
        const int last = min(u.tok0 + (w + 1) * kRows, x.T);   // behind the warpgroup's last token
        const int end = p.causal ? max(0, x.N - x.T + last) : x.N;
        u.tiles[w] = last > u.tok0 + w * kRows ? (end + kTile - 1) / kTile : -1;
        if (u.tiles[w] >= 0) u.end = end;
    }
}
// By every thread; scratch: kSorted int2, and a word.
__device__ inline void sort_blocks(const LatentPrefillParams& p, Smem& s, uint8_t* scratch) {
    int2* found = reinterpret_cast<int2*>(scratch);
    int* count = reinterpret_cast<int*>(scratch + kSorted * sizeof(int2));
    if (threadIdx.x == 0) *count = 0;
    __syncthreads();
    for (int b = threadIdx.x; b < p.B; b += kThreads) {
        const Span x = load_span(p, b, blockIdx.x == 0);
        const int n = x.blocks();
        if (n == 0) continue;
        const int at = atomicAdd(count, min(n, kSorted + 1));
        for (int i = 0; i < n && at + i < kSorted; ++i) found[at + i] = make_int2(block_end(p, x, i), b << kBlockBits | i);
    }
    __syncthreads();
    const int n = *count;
    if (threadIdx.x == 0) s.sorted = n <= kSorted ? n : -1;
    for (int i = threadIdx.x; n <= kSorted && i < n; i += kThreads) {   // (equal ones by request and block, however they came)
        const int2 x = found[i];
        int rank = 0;
        for (int k = 0; k < n; ++k) rank += found[k].x > x.x || (found[k].x == x.x && found[k].y > x.y);
        s.order[rank] = x.y;
    }
    __syncthreads();
}
struct Units {
    int64_t before;   // units of requests before lane 0's
    int b0;
    int64_t up;       // units up to this lane's request, itself included
    Span x;
    __device__ __forceinline__ void load(const LatentPrefillParams& p, int lane) {
        const int b = b0 + lane;
        x = b < p.B ? load_span(p, b, false) : Span{0, 0, 0, 0};
        up = static_cast<int64_t>(x.blocks()) * p.n_q;
        #pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(kFull, up, o);
            if (lane >= o) up += v;
        }
        up += before;
    }
    // Unit u (not before the last one asked for); false behind the last.
    __device__ __forceinline__ bool find(const LatentPrefillParams& p, const Smem& s, int64_t u, int lane, Unit& out) {
        if (s.sorted >= 0) {
            if (u >= static_cast<int64_t>(s.sorted) * p.n_q) return false;
            const uint32_t e = s.order[u / p.n_q];
            const int b = static_cast<int>(e >> kBlockBits);
            make_unit(p, load_span(p, b, false), b, static_cast<int>(u % p.n_q), static_cast<int>(e & ((1u << kBlockBits) - 1)), out);
            return true;
        }
        while (true) {
            const unsigned at = __ballot_sync(kFull, u < up);
            if (at) {
                const int src = __ffs(at) - 1;
                const int64_t prev = __shfl_sync(kFull, up, src > 0 ? src - 1 : 0), in = u - (src > 0 ? prev : before);
                const Span y{__shfl_sync(kFull, x.s0, src), __shfl_sync(kFull, x.T, src), __shfl_sync(kFull, x.k0, src), __shfl_sync(kFull, x.N, src)};
                make_unit(p, y, b0 + src, static_cast<int>(in % p.n_q), y.blocks() - 1 - static_cast<int>(in / p.n_q), out);
                return true;
            }
            before = __shfl_sync(kFull, up, 31);
            b0 += 32;
            if (b0 >= p.B) return false;
            load(p, lane);
        }
    }
};

__device__ __forceinline__ void producer(Smem& s, const LatentPrefillParams& p, const Maps& m, int lane) {
    Units units;
    units.before = 0;
    units.b0 = 0;
    if (s.sorted < 0) units.load(p, lane);
    uint32_t n = 0, pieces = 0, done[2] = {0, 0};   // tiles before; pieces asked for; units with rows of each warpgroup
    bool ok = true;
    #pragma unroll 1
    for (uint32_t i = 0;; ++i) {
        const int64_t turn = static_cast<int64_t>(i) * gridDim.x;
        Unit x;
        const bool more = units.find(p, s, turn + (i & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x), lane, x);
        // (a turn that is cut off may lack this CTA's unit: so does every later one)
        const uint32_t at = i & 1;
        ok = i < 2 || wait_bar(s, &s.u_empty[at], i / 2 - 1);
        if (!ok) break;
        if (lane == 0) {
            if (!more) x.b = -1;
            x.turn[0] = done[0];
            x.turn[1] = done[1];
            s.unit[at] = x;
            mbar_arrive(&s.u_full[at]);
        }
        __syncwarp();
        if (!more) break;
        const int tiles = max(x.tiles[0], x.tiles[1]);
        #pragma unroll
        for (int w = 0; w < 2; ++w) {
            if (x.tiles[w] <= 0 || !ok) continue;
            if (done[w]) ok = wait_bar(s, &s.q_empty[w], done[w] - 1);
            if (!ok) continue;
            ++done[w];
            if (lane == 0) {
                mbar_arrive_expect_tx(&s.q_full[w], 3 * kChunk);
                for (int c = 0; c < 3; ++c) tma3(s.q[w] + c * kChunk, &m.q, c * 64, x.h, x.s0 + x.tok0 + w * kRows, &s.q_full[w]);
            }
            __syncwarp();
        }
        #pragma unroll 1
        for (int t = 0; ok && t < tiles; ++t, ++n) {
            const int key = x.k0 + t * kTile;
            #pragma unroll 1
            for (int k = 0; k < kTilePieces; ++k) {
                const uint32_t piece = n * kTilePieces + k, at = piece % kPieces;
                if (piece >= kPieces) ok = wait_bar(s, &s.empty[at], piece / kPieces - 1);
                if (!ok) break;
                pieces = piece + 1;
                if (lane == 0) {
                    mbar_arrive_expect_tx(&s.full[at], kPieceBytes);
                    if (k < 2) {
                        tma3(s.piece[at], &m.k, k * 64, x.h, key, &s.full[at]);
                    } else if (k == 2) {
                        tma2(s.piece[at], &m.r, 0, key, &s.full[at]);
                    } else {
                        tma3(s.piece[at], &m.v, 0, x.h, key + (k - 3) * 64, &s.full[at]);
                        tma3(s.piece[at] + kPieceBytes / 2, &m.v, 64, x.h, key + (k - 3) * 64, &s.full[at]);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok) break;
    }
    if (s.abort) {   // copies under way must land in memory that is still this block's
        for (uint32_t k = pieces > kPieces ? pieces - kPieces : 0; k < pieces; ++k) mbar_wait(&s.full[k % kPieces], (k / kPieces) & 1u, nullptr, kWaitNs);
        for (int w = 0; w < 2; ++w)
            if (done[w]) mbar_wait(&s.q_full[w], (done[w] - 1) & 1u, nullptr, kWaitNs);
    }
}

// The unit's description, by every role in turn; false behind the last.
__device__ __forceinline__ bool next_unit(Smem& s, uint32_t i, Unit& x, int lane) {
    if (!wait_bar(s, &s.u_full[i & 1], i / 2)) return false;
    x = s.unit[i & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.u_empty[i & 1]);
    return x.b >= 0;
}

// --------------------------------------------------------------------- issue
// V as it is in memory: 64 dims a row of 128 bytes, groups of eight keys 1,024 bytes apart, the other 64 dims behind them.
__device__ __forceinline__ uint64_t desc_v(uint32_t addr) {
    return static_cast<uint64_t>(addr >> 4) | (static_cast<uint64_t>(kPieceBytes / 2 >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}

// A warp for each softmax warpgroup: O(t) += P(t)·V(t), then S(t + 1) = Q·K(t + 1)ᵀ over the P that has been read.  One warp for
// both left the tensor cores idle for half of the time: what stands between two runs of MMAs (waits, descriptors, commits)
// takes 500 to 700 cycles, a run 520 or 780, and few MMAs are taken ahead.  The two take turns: mixed, their MMAs end at the
// same time, and both warpgroups' softmax runs while the tensor cores have nothing to do.
// Every operand is a value that all lanes have, and known as one: an instruction then issues in its own time.
template <bool TWO>
__device__ __forceinline__ void issuer(Smem& s, int w, int lane) {
    constexpr uint32_t kDescS = mma_desc_bf16(kRows, kTile), kDescO = mma_desc_bf16(kRows, kExpVal) | (1u << 16);
    const uint32_t W = uniform(w), tmem = uniform(s.tmem), p_op = uniform(smem_u32(s.piece));
    const uint32_t q_op = uniform(smem_u32(s.q) + W * 3 * kChunk), col_s = uniform(tmem + kColS + W * kTile), col_o = uniform(tmem + kColO + W * kExpVal);
    Unit x;
    uint32_t n = 0, units = 0, steps = 0;
    bool ok = true;
    auto place = [&](uint32_t piece) { return uniform(p_op + piece % kPieces * kPieceBytes); };
    auto barrier = [&](uint32_t piece) { return uniform(smem_u32(&s.empty[piece % kPieces])); };
    auto wait_piece = [&](uint32_t piece) { return wait_bar(s, &s.full[piece % kPieces], piece / kPieces); };
    auto commit = [&](uint64_t* bar) {
        const uint32_t b = uniform(smem_u32(bar));
        if (elect_one()) mma_commit(b);
        __syncwarp();
    };
    const uint32_t s_full = uniform(smem_u32(&s.s_full[W]));
    struct Keys {
        uint32_t b[3], e[3];
    };
    auto keys_of = [&](uint32_t t) {   // of the CTA's tile t
        const uint32_t piece = t * kTilePieces;
        return Keys{{place(piece), place(piece + 1), place(piece + 2)}, {barrier(piece), barrier(piece + 1), barrier(piece + 2)}};
    };
    // S of the CTA's tile t; `last` of the unit's: Q has been read.  With the turn, which goes while K is not there yet: K may
    // want a place that the other warpgroup's product with V has to leave first.
    auto scores = [&](uint32_t t, const Keys& k, bool last) {
        const uint32_t piece = t * kTilePieces + min(lane, 2);
        uint64_t* bar = lane < 3 ? &s.full[piece % kPieces] : nullptr;
        if (!test_lanes(bar, piece / kPieces)) {
            give_turn(s, lane);
            ok = wait_lanes(s, bar, piece / kPieces) && take_turn(s, lane);
            if (!ok) return;
        }
        tcgen_fence_after();
        auto chunk = [&](int c) {
            #pragma unroll
            for (int i = 0; i < 4; ++i)
                mma_ss(col_s, smem_desc_sw128(q_op + c * kChunk + i * 32), smem_desc_sw128(k.b[c] + i * 32), kDescS, (c | i) != 0);
        };
        if (elect_one()) {
            chunk(0);
            mma_commit(k.e[0]);
            chunk(1);
            mma_commit(k.e[1]);
        }
        give_turn(s, lane);   // the other one comes while the rest runs
        if (elect_one()) {
            chunk(2);
            mma_commit(s_full);
            mma_commit(k.e[2]);
        }
        __syncwarp();
        if (last) commit(&s.q_empty[W]);
    };
    while (ok && next_unit(s, units, x, lane)) {
        const uint32_t mine = uniform(max(x.tiles[W], 0)), tiles = uniform(max(max(x.tiles[0], x.tiles[1]), 0));
        if (mine > 0) {
            const Keys keys = keys_of(n);
            ok = wait_bar(s, &s.q_full[W], x.turn[W]) && take_turn(s, lane);
            if (ok) scores(n, keys, mine == 1);
        }
        #pragma unroll 1
        for (uint32_t t = 0; ok && t < mine; ++t) {
            const uint32_t piece = (n + t) * kTilePieces + 3;
            const uint32_t b[2] = {place(piece), place(piece + 1)}, e[2] = {barrier(piece), barrier(piece + 1)}, add = uniform(t > 0);
            const Keys keys = keys_of(n + t + 1);
            const uint32_t other = piece + (lane == 2);
            ok = wait_lanes(s, lane == 0 ? &s.p_full[W] : lane < 3 ? &s.full[other % kPieces] : nullptr, lane == 0 ? steps : other / kPieces) &&
                 take_turn(s, lane);
            if (!ok) break;
            ++steps;
            tcgen_fence_after();
            if (elect_one()) {
                #pragma unroll
                for (int half = 0; half < 2; ++half) {
                    #pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        mma_ts(col_o, col_s + (half * 4 + k) * 8, desc_v(b[half] + k * 2048), kDescO, half > 0 || k > 0 ? 1u : add);
                        if (TWO) mma_ts(col_o, col_s + kColRest + (half * 4 + k) * 8, desc_v(b[half] + k * 2048), kDescO, 1u);
                    }
                    mma_commit(e[half]);
                }
            }
            __syncwarp();
            if (t + 1 < mine) {
                scores(n + t + 1, keys, t + 2 == mine);
            } else {
                give_turn(s, lane);
                commit(&s.o_full[W]);
            }
        }
        for (uint32_t k = (n + mine) * kTilePieces; ok && k < (n + tiles) * kTilePieces; ++k) {   // of the other warpgroup's rows alone
            ok = wait_piece(k);
            if (ok && lane == 0) mbar_arrive(&s.empty[k % kPieces]);
            __syncwarp();
        }
        n += tiles;
        ++units;
    }
    // the last commits arrive in this block's shared memory, and nothing is under way in tensor memory
    commit(&s.drain[W]);
    mbar_wait(&s.drain[W], 0, nullptr, kWaitNs);
    if (!s.abort)
        for (uint32_t k = n * kTilePieces > kPieces ? n * kTilePieces - kPieces : 0; k < n * kTilePieces; ++k)
            if (!wait_bar(s, &s.empty[k % kPieces], k / kPieces)) break;
}

// 32 bytes, a whole sector of a row that no other thread writes to, if they stand on one.
__device__ __forceinline__ void st32(void* p, const uint32_t* v, bool sector) {
    if (sector) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]),
                     "r"(v[5]), "r"(v[6]), "r"(v[7])
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// ------------------------------------------------------------------- softmax
// What two weights' upper 16 bits leave of them, as two bf16, and 2^-23 of them more: above 0 wherever a weight is (one of 2^-102 or
// more), so that an infinite value times either part has the value's sign.  (By a minimum and a maximum, which have no such border, a prompt of
// 8,192 takes 699 us, by packed ones 665.)
__device__ __forceinline__ uint32_t rests_of(float2 a, uint32_t x, uint32_t y) {
    const float c = 1.f + 0x1p-23f;
    const float2 d = fma2(a, make_float2(c, c), make_float2(__uint_as_float((x & 0xffff0000u) ^ 0x80000000u), __uint_as_float((y & 0xffff0000u) ^ 0x80000000u)));
    return pack_bf16(d.x, d.y);
}
template <bool TWO>
__device__ __forceinline__ void softmax(Smem& s, const LatentPrefillParams& p, int w, int tid, int lane) {
    const uint32_t mine = s.tmem + (static_cast<uint32_t>(tid & ~31) << 16);
    const uint32_t col_s = mine + kColS + w * kTile, col_o = mine + kColO + w * kExpVal;
    const bool negative = p.scale_log2 < 0.f;
    const float scale = p.scale_log2 == 0.f ? 1e-38f : fabsf(p.scale_log2);   // (0·−inf of a masked key would be NaN)
    const bool sector = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    Unit x;
    uint32_t n = 0, all = 0, units = 0;   // tiles before, of this warpgroup and of the CTA
    for (uint32_t i = 0; next_unit(s, i, x, lane); ++i) {
        const int tiles = max(x.tiles[0], x.tiles[1]);
        const uint32_t before = all;
        all += max(tiles, 0);
        if (x.tiles[w] < 0) continue;
        const int r = x.tok0 + w * kRows + tid;               // token of the request
        const int last = p.causal ? x.N - x.T + r : x.N - 1;   // the last key it attends
        const int first = p.causal ? x.N - x.T + x.tok0 + w * kRows : x.N - 1;   // of the warpgroup's first row
        float ref = -INFINITY;
        float2 sum = make_float2(0.f, 0.f);
        #pragma unroll 1
        for (int t = 0; t < x.tiles[w]; ++t, ++n) {
            if (!wait_bar(s, &s.s_full[w], n)) return;   // (the product with V before it is done as well)
            tcgen_fence_after();
            uint32_t v[4][32];
            #pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(col_s + c * 32, v[c]);
            #pragma unroll
            for (int c = 0; c < 4; ++c) tmem_wait_ld(v[c]);
            if (negative) {
                #pragma unroll
                for (int c = 0; c < 4; ++c)
                    #pragma unroll
                    for (int e = 0; e < 32; ++e) v[c][e] ^= 0x80000000u;
            }
            const int base = t * kTile;
            if (base + kTile - 1 > min(first, x.N - 1)) {
                const int keep = min(last, x.N - 1) - base;   // columns up to this one
                #pragma unroll
                for (int c = 0; c < 4; ++c)
                    #pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (c * 32 + e > keep) v[c][e] = 0xff800000u;
            }
            float top[4];
            #pragma unroll
            for (int c = 0; c < 4; ++c) {
                top[c] = max3(__uint_as_float(v[c][0]), __uint_as_float(v[c][1]), __uint_as_float(v[c][2]));
                #pragma unroll
                for (int e = 3; e < 31; e += 2) top[c] = max3(top[c], __uint_as_float(v[c][e]), __uint_as_float(v[c][e + 1]));
                top[c] = fmaxf(top[c], __uint_as_float(v[c][31]));
            }
            const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * scale;
            const bool moved = most > ref + kLazy;
            if (__any_sync(kFull, moved)) {
                const float f = moved ? ex2(ref - most) : 1.f;
                if (moved) ref = most;
                sum = mul2(sum, make_float2(f, f));
                if (t > 0) {
                    #pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t o[32];
                        tmem_ld32(col_o + c * 32, o);
                        tmem_wait_ld(o);
                        #pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                        tmem_st32(col_o + c * 32, o);
                    }
                }
            }
            if (t == tiles - 1 && x.end < base + kTile) {
                // V behind the last key that a row of the unit attends: its weight is 0, and 0·NaN would be NaN.  Each warpgroup with
                // rows there does it before its own p_full: nothing else orders the other's stores before its product.  (Zeros over
                // zeros the second time, in a piece that stays until this warpgroup's issuer has released it too.)
                #pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const uint32_t piece = (before + t) * kTilePieces + 3 + half, at = piece % kPieces;
                    if (!wait_bar(s, &s.full[at], piece / kPieces)) return;
                    for (int c = max(x.end - base - half * 64, 0) + (tid >> 4); c < 64; c += 8)
                        *reinterpret_cast<uint4*>(s.piece[at] + (tid >> 3 & 1) * (kPieceBytes / 2) + c * 128 + (tid & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_shared();
            }
            const float z = ref == -INFINITY ? 0.f : -ref;
            constexpr int kStep = TWO ? 1 : 2;   // (16 registers of each at a time: 32 spill)
            #pragma unroll
            for (int c = 0; c < 4; c += kStep) {
                uint32_t pk[16 * kStep], rest[16];
                #pragma unroll
                for (int e = 0; e < 16 * kStep; ++e) {
                    float2 a = make_float2(__uint_as_float(v[c + (e >> 4)][2 * (e & 15)]), __uint_as_float(v[c + (e >> 4)][2 * (e & 15) + 1]));
                    a = fma2(a, make_float2(scale, scale), make_float2(z, z));
                    a.x = ex2(a.x);
                    a.y = ex2(a.y);
                    sum = add2(sum, a);
                    if constexpr (TWO) {
                        const uint32_t x = __float_as_uint(a.x), y = __float_as_uint(a.y);
                        pk[e] = __byte_perm(x, y, 0x7632);
                        rest[e] = rests_of(a, x, y);
                    } else {
                        pk[e] = pack_bf16(a.x, a.y);
                    }
                }
                if constexpr (TWO) {
                    tmem_st16(col_s + c * 16, pk);
                    tmem_st16(col_s + kColRest + c * 16, rest);
                } else {
                    tmem_st32(col_s + c * 16, pk);
                }
            }
            tmem_wait_st();
            tcgen_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.p_full[w]);
        }
        const float total = sum.x + sum.y, inv = total == 0.f ? 0.f : 1.f / total;
        const bool real = r < x.T;
        const int64_t row = (static_cast<int64_t>(x.s0) + r) * p.n_q + x.h;
        const bool any = x.tiles[w] > 0;
        if (any) {
            if (!wait_bar(s, &s.o_full[w], units++)) return;
            tcgen_fence_after();
        }
        float odd = 0.f;
        #pragma unroll 1
        for (int c = 0; c < 4; ++c) {
            uint32_t o[32];
            if (any) {
                tmem_ld32(col_o + c * 32, o);
                tmem_wait_ld(o);
            } else {
                #pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = 0;
            }
            float y[32];
            #pragma unroll
            for (int e = 0; e < 32; ++e) {
                y[e] = __uint_as_float(o[e]) * inv;
                odd += y[e];
            }
            if (!real) continue;
            if constexpr (TWO) {
                uint32_t z[32];
                #pragma unroll
                for (int e = 0; e < 32; ++e) z[e] = __float_as_uint(y[e]);
                #pragma unroll
                for (int e = 0; e < 32; e += 8) st32(static_cast<float*>(p.out) + row * kExpVal + c * 32 + e, z + e, sector);
            } else {
                uint32_t z[16];
                #pragma unroll
                for (int e = 0; e < 16; ++e) z[e] = pack_bf16(y[2 * e], y[2 * e + 1]);
                #pragma unroll
                for (int e = 0; e < 16; e += 8) st32(static_cast<uint16_t*>(p.out) + row * kExpVal + c * 32 + 2 * e, z + e, sector);
            }
        }
        if (real && p.lse_out) p.lse_out[row] = total == 0.f ? -INFINITY : (ref + log2f(total)) * kLn2;
        tcgen_fence_before();
        // A key that some rows of a tile attend and others do not may hold what is not finite: its weight is 0 for those,
        // and 0·NaN is NaN.  A row that came out as NaN is computed again if its tiles hold such a key behind what it attends (else
        // it is NaN by right).
        unsigned todo = __ballot_sync(kFull, p.causal && real && odd != odd);
        for (; todo; todo &= todo - 1) {
            const int rr = (r & ~31) + __ffs(todo) - 1, end = max(0, x.N - x.T + rr + 1);
            __syncwarp();
            if (!odd_values(p, x.h, x.k0, end, min(x.tiles[w] * kTile, x.end))) continue;
            if (lane == 0) atomicAdd(&s.again, 1);
            plain_row(p, static_cast<int64_t>(x.s0) + rr, x.h, x.k0, end);
            if (lane == 0) atomicSub(&s.again, 1);
        }
    }
}

template <bool TWO>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const LatentPrefillParams p, const __grid_constant__ Maps m) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    Smem& s = *reinterpret_cast<Smem*>(smem_raw);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == kIssueWarp) tmem_alloc_all(&s.tmem);
    if (tid == 0) {
        for (int i = 0; i < kPieces; ++i) {
            mbar_init(&s.full[i], 1);
            mbar_init(&s.empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s.drain[i], 1);
            mbar_init(&s.q_full[i], 1);
            mbar_init(&s.q_empty[i], 1);
            mbar_init(&s.s_full[i], 1);
            mbar_init(&s.p_full[i], 4);
            mbar_init(&s.o_full[i], 1);
            mbar_init(&s.u_full[i], 1);
            mbar_init(&s.u_empty[i], kReaders);
        }
        mbar_fence_init();
        s.turn = 0;
        s.abort = 0;
        s.again = 0;
    }
    pdl_wait();
    pdl_trigger();
    sort_blocks(p, s, s.piece[0]);
    fence_proxy_async_shared();   // the scratch is copied over
    tcgen_fence_before();
    __syncthreads();
    tcgen_fence_after();
    // the operands' swizzle wants 1,024-byte addresses (nothing else stands before them)
    const bool aligned = (smem_u32(smem_raw) & 1023u) == 0;
    if (!aligned && tid == 0) report(p.err, KVD_ERR_CUDA);
    // a thread has 168 registers at launch: 2·208 + 80 = 496 ≤ 3·168
    if (aligned) {
        if (warp < 8) {
            take_registers<208>();
            softmax<TWO>(s, p, warp >> 2, tid & 127, lane);
        } else {
            give_registers<80>();
            if (warp == kProducerWarp) producer(s, p, m, lane);
            else if (warp == kIssueWarp || warp == kIssueWarp + 1) issuer<TWO>(s, warp - kIssueWarp, lane);
        }
    }
    __syncwarp();
    tcgen_fence_before();
    __syncthreads();
    tcgen_fence_after();
    if (warp == kIssueWarp) {
        if (lane == 0 && s.abort) report(p.err, KVD_ERR_TIMEOUT);
        tmem_free_all(s.tmem);
    }
}

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
Encode encoder() {
    static const Encode fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<Encode>(f);
    }();
    return fn;
}

// [rows][heads][dims] bf16 (heads 0: [rows][dims]), copied 64 dims of one head and `box` rows at a time; rows behind the
// last are read as zeros.
bool make_map(CUtensorMap* map, const void* base, int dims, int heads, int64_t rows, int64_t head_stride, int64_t stride, int box) {
    cuuint64_t size[3] = {static_cast<cuuint64_t>(dims)}, pitch[2];
    cuuint32_t tile[3] = {64}, step[3] = {1, 1, 1};
    int rank = 1;
    if (heads > 0) {
        pitch[rank - 1] = static_cast<cuuint64_t>(2 * head_stride);
        size[rank] = static_cast<cuuint64_t>(heads);
        tile[rank++] = 1;
    }
    pitch[rank - 1] = static_cast<cuuint64_t>(2 * stride);
    size[rank] = static_cast<cuuint64_t>(rows);
    tile[rank++] = static_cast<cuuint32_t>(box);
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, static_cast<cuuint32_t>(rank), const_cast<void*>(base), size, pitch, tile, step,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_latent_prefill(const LatentPrefillParams& p, int num_sms, cudaStream_t stream) {
    static_assert(sizeof(Smem) <= 232448, "shared memory of one SM");
    Maps m;
    if (!encoder()) return cudaErrorNotSupported;
    // without keys no unit has a tile, and no map but a valid one is needed
    const bool keys = p.n_keys > 0;
    const void* any = p.q;
    if (!make_map(&m.q, p.q, kExpKey, p.n_q, p.n_tokens, kExpKey, static_cast<int64_t>(p.n_q) * kExpKey, kRows) ||
        !make_map(&m.k, keys ? p.k_nope : any, kNope, p.n_q, keys ? p.n_keys : 1, keys ? p.k_head : kNope, keys ? p.k_stride : kNope * p.n_q, kTile) ||
        !make_map(&m.v, keys ? p.v : any, kExpVal, p.n_q, keys ? p.n_keys : 1, keys ? p.v_head : kExpVal, keys ? p.v_stride : kExpVal * p.n_q, 64) ||
        !make_map(&m.r, keys ? p.k_rope : any, kLatRope, 0, keys ? p.n_keys : 1, 0, keys ? p.rope_stride : kLatRope, kTile))
        return cudaErrorInvalidValue;
    auto* kernel = p.out_f32 ? prefill_kernel<true> : prefill_kernel<false>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(Smem)));
    if (e != cudaSuccess) return e;
    return launch_dependent(kernel, dim3(static_cast<unsigned>(num_sms)), dim3(kThreads), sizeof(Smem), -1, stream, p, m);
}

}  // namespace kvd
