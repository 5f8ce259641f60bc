// attn_pair.cuh -- tile sizes, shared-memory layout, barriers and register split
// of the CTA-pair attention kernels (attn_tc.cu: packed KV rows; attn_paged.cu:
// a paged cache).  The algorithm is described at the top of attn_tc.cu.
#pragma once
#include "dsa_kernels.h"

namespace dsa {

// Exchange layout of the partial scores and of P: 16-byte chunk c (4 fp32
// partials, or 8 bf16 probabilities) of head row h at c*2048 + h*16.  A warp's
// stores of one chunk then cover 512 contiguous bytes, which the cluster's
// shared-memory path moves several times faster than 32 scattered 16-byte
// pieces; for P it is also the no-swizzle K-major operand layout of the MMA
// (8-row x 16-byte core matrices, 128 B apart along M and 2048 B along K).
__device__ __forceinline__ uint32_t chunk_off(int h, int c) { return (uint32_t)(c * 2048 + h * 16); }
#ifndef DSA_ATTN_EPI_STAGE
#define DSA_ATTN_EPI_STAGE 1
#endif
constexpr int AT_N = 64;                           // keys per tile
constexpr uint32_t AT_BLK = AT_N * 128;            // one 64-column block of a tile
constexpr uint32_t AT_KST = 5 * AT_BLK;            // K part of a stage (max 5 blocks)
constexpr uint32_t AT_VST = 4 * AT_BLK;            // V part (separate V only)
constexpr uint32_t AT_TILE128 = 128 * 128;         // a 128-row x 128-byte tile
constexpr uint32_t AT_SX_BYTES = 128 * 128 + 128 * 4;  // partial scores + partial maxima
constexpr uint32_t AT_PX_BYTES = 128 * 64;         // the peer's half of P
constexpr uint32_t AT_LX_BYTES = 128 * 4;          // the peer's row sums
constexpr uint32_t TM_O = 0, TM_S = 256, TM_Q = 384;  // S: two 64-column partial accumulators
constexpr int AT_THREADS = 512;  // 6 producer + 2 MMA + 8 softmax warps
constexpr int AT_PRODUCERS = 6;
constexpr int AT_MMA2_WARP = 6;  // issues the second half of every S tile
constexpr int AT_MMA_WARP = 7;
constexpr int AT_SOFT0 = 8;      // first softmax warp (a warpgroup boundary)
// Register split (setmaxnreg): warpgroup 0 (producers 0-3) and warpgroup 1
// (producers 4-5 and the two MMA warps) give registers to the softmax
// warpgroups.  setmaxnreg.inc draws only on the registers the block was
// launched with, so the split must fit the launch total (threads x registers
// per thread at launch), or the softmax warps wait forever; the launcher
// checks the compiled count before every launch.
constexpr int AT_REGS_WG0 = 40;
constexpr int AT_REGS_WG1 = 56;
constexpr int AT_REGS_SOFT = 208;
constexpr int AT_REGS_SPLIT = 128 * AT_REGS_WG0 + 128 * AT_REGS_WG1 + (AT_THREADS - 256) * AT_REGS_SOFT;
static_assert(AT_SOFT0 == 8, "the register split assumes two producer/MMA warpgroups");
static_assert(AT_REGS_SPLIT <= ((65536 / AT_THREADS) & ~7) * AT_THREADS, "register split above the launch total");
constexpr int AT_SCAN_ROUNDS = (2048 / 32 + AT_PRODUCERS - 1) / AT_PRODUCERS;  // index-row words per producer warp
constexpr int AT_NTAB = 8;       // tile counts of the queries between the PV and the S cursor

template <int NST, bool VSEP, int NPB = 2, int NSX = 1>
struct AtLayout {
    static constexpr uint32_t STAGE = AT_KST + (VSEP ? AT_VST : 0);
    static constexpr uint32_t OFF_QR = NST * STAGE;               // rank 1's 5th Q block (rope), A of SS MMAs
    static constexpr uint32_t OFF_P = OFF_QR + AT_TILE128;        // [NPB] P tiles
    static constexpr uint32_t OFF_SX = OFF_P + NPB * AT_TILE128;  // [NSX] partial-score tiles
    static constexpr uint32_t OFF_PM = OFF_SX + NSX * AT_TILE128; // [NSX][128] partial maxima
    static constexpr uint32_t OFF_LX = OFF_PM + NSX * 512;        // [128] combined row sums (B -> A warps)
    static constexpr uint32_t OFF_LXR = OFF_LX + 512;             // [128] the peer's row sums
    static constexpr uint32_t OFF_VM = OFF_LXR + 512;             // [2][64] validity bits of 2048 slots
    static constexpr uint32_t OFF_INFO = OFF_VM + 512;            // [2][8] last used slot per producer warp, [8] tile counts
    static constexpr uint32_t OFF_BAR = OFF_INFO + 128;
    // epilogue staging: per softmax warp 32 rows x 64 output columns (bf16),
    // so that the output stores cover whole 128-byte lines; with three P
    // tiles, 32 rows x 32 columns (64-byte segments) to make room
    static constexpr bool EPI_STAGE = !VSEP && DSA_ATTN_EPI_STAGE;
    static constexpr int EPI_COLS = NPB >= 3 ? 32 : 64;
    static constexpr uint32_t EPI_WARP_BYTES = 32 * EPI_COLS * 2;
    static constexpr uint32_t OFF_EPI = OFF_BAR + 512;
    static constexpr uint32_t SMEM = OFF_EPI + (EPI_STAGE ? 8 * EPI_WARP_BYTES : 0);
};

struct AtBars {
    uint64_t full[4];
    uint64_t empty[4];
    uint64_t s_full, s_empty;  // the S tile (both issuers committed) / read by the 8 softmax warps
    uint64_t s_go;             // the second issuer may issue its half of the next S tile
    uint64_t q_full;         // Q of the next query with tiles is in place (4 A warps)
    uint64_t o_full;         // all PVs of a query done
    uint64_t o_free;         // its epilogue has read O (8 softmax warps)
    uint64_t p_full[3];      // 4 local B warps + the peer's half of P (bytes)
    uint64_t p_free[3];      // PV done in both CTAs (multicast commit)
    uint64_t sx_full[2];     // the peer's partial scores (bytes)
    uint64_t sx_free[2];     // the peer consumed the partials this CTA sent
    uint64_t lx_full;        // the peer's row sums (bytes)
    uint64_t lx_loc;         // the B warps combined the row sums (for the A warps)
    uint64_t drain;
    uint64_t info_full[2];   // query info published (7 producer warps)
    uint64_t info_empty[2];  // query info consumed (MMA warp + 8 softmax warps)
    uint64_t drain2;
    int go[2];  // stage of the S tile announced on s_go, -1: no more tiles
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(AtBars) <= 512, "barrier block");

__device__ __forceinline__ uint32_t swz(int row, int chunk) { return (uint32_t)(row * 128 + ((chunk ^ (row & 7)) << 4)); }

}  // namespace dsa
