/*
 * mmq.h -- C ABI of the GB300 (sm_103a) prefill quantized matrix multiply (MMQ):
 * k-quant weight super-blocks (q6_K 210 B, q4_K 144 B, 256 values each) times
 * per-32 q8 activations,
 *
 *     q6_K: Y[t,j] = sum_c sum_h d_a[t,c] * (d*sc[2(c%8)+h]) * I[t,j,c,h]
 *     q4_K: Y[t,j] = sum_c d_a[t,c] * ((d*sc_c) * I[t,j,c] - (dmin*m_c) * ssum[t,c])
 *
 * (d, sc, dmin, m from the weight super-block; d_a, ssum the activation chunk's
 * scale and code sum)
 *
 * with I the integer dot of a 16-value (q6_K) or 32-value (q4_K) sub-block.
 *
 * Sources (page title, section):
 *   [r45] "r45 - cp.async for the q6_K A-side staging: mechanism confirmed,
 *          wall-neutral (REVERTED)"
 *   [r56] "r56 - q6_K A-side bundle: A cp.async + W_dsc f32 plane (LANDED)"
 *   [r58] "r58 - q4_K BT spec + cp.async-db2 transplant (REVERTED)"
 * The pages show the registration step, the activation prepass and the GEMM
 * launch ([r56] §3.1: registration gates and planes; [r45] §1.1: the
 * quantize-transpose prepass; [r58] §2.2: the GEMM's staging); this ABI exposes
 * those three steps as calls.
 *
 * Conventions (all calls):
 *  - Every buffer pointer is a DEVICE pointer owned by the caller.  The library
 *    never allocates or frees device memory; sizes come from the *_bytes queries.
 *  - Calls are asynchronous on stream `s` (NULL = legacy default stream).
 *    Argument, shape and alignment errors are returned synchronously, before
 *    anything is launched; a failed launch returns MMQ_ERR_CUDA.
 *  - K = id must be a multiple of 256 (one super-block); od >= 1 may be odd; M >= 1.
 *  - Buffers read by bulk copies (qa, scales, packed) must be 16-byte aligned,
 *    else MMQ_ERR_ALIGN.  x and Y need 4-byte alignment.
 *  - Every bounded wait inside a kernel gives up after about two seconds, sets the
 *    library's one sticky device error word for waits (one per device) and lets the kernel
 *    exit; mmq_get_device_error() reports and clears it, whichever kernel set it.
 *    Results of a launch that timed out are undefined, and so are those of launches
 *    queued after it until the word is cleared (their waits give up early once they
 *    see it set).
 *  - Calls may come from several host threads; the one piece of shared host
 *    state is the label mmq_last_path() returns (the most recent GEMM launch
 *    of the process).
 */
#ifndef MMQ_GB300_H
#define MMQ_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t (the runtime's stream handle). */
typedef struct CUstream_st* mmq_stream_t;

typedef enum {
    MMQ_OK = 0,
    MMQ_ERR_ARG = 1,         /* null pointer, bad type id, ldx < K, ldy < od */
    MMQ_ERR_SHAPE = 2,       /* K/id not a multiple of 256, M/od < 1, sizes over the limits */
    MMQ_ERR_ALIGN = 3,       /* a pointer is not aligned as stated above */
    MMQ_ERR_CUDA = 4,        /* a CUDA runtime call or launch failed */
    MMQ_ERR_TIMEOUT = 5,     /* a bounded in-kernel wait expired (see mmq_get_device_error) */
    MMQ_ERR_UNSUPPORTED = 6  /* no sm_103 device is current */
} mmq_status;

typedef enum { MMQ_Q4_K = 12, MMQ_Q6_K = 14 } mmq_type;

/* Size limits (checked; MMQ_ERR_SHAPE beyond them). */
#define MMQ_MAX_M (1 << 22)
#define MMQ_MAX_OD (1 << 22)
#define MMQ_MAX_ID (1 << 20)

/* --------------------------------------------------------------------------
 * Activation planes ([r45] §2.3 and [r56] §1: the prepass writes a
 * pre-transposed q8 code plane and a d/ssum scale pair per (chunk, token),
 * padded token rows zero-filled).
 *
 * Layout (fixed, documented so a caller can read it back):
 *   Mp = 128 * ceil(M/128) padded tokens; nkb = K/64; nchunk = K/32; nsb = K/256.
 *   qa:     Mp*K f16 values, the q8 codes held as exact binary16 integers
 *           (zero as +0).
 *           Tile (mt, kb) = tokens 128*mt.. and values 64*kb.. is a 16384-byte
 *           block at byte (mt*nkb + kb)*16384.  Inside it token r (0..127) and
 *           value k (0..63) sit at byte r*128 + (((k/8) ^ (r%8))*16) + (k%8)*2
 *           (the 128-byte swizzle of the tensor-core operand tile).
 *   scales: two planes (offsets from mmq_act_scale_layout):
 *     pairs  Mp*nchunk entries of 8 bytes {float d, int32 ssum}; entry (t, c) at
 *            index ((t/128)*nchunk + c)*128 + t%128.
 *     am     the q4_K min-term operand ma = d*ssum (one f32 multiply) split into
 *            tf32 hi = round-to-nearest(ma) and lo = round-to-nearest(ma - hi):
 *            per (token tile mt, super-block sb) an 8192-byte block at
 *            (mt*nsb + sb)*8192 holding the hi tile then the lo tile, each
 *            128 rows x 8 chunks of 4-byte values, row r / chunk k at byte
 *            (r/8)*256 + (k/4)*128 + (r%8)*16 + (k%4)*4.
 *   Rows t >= M hold code 0, d 0, ssum 0, ma 0.
 *   qa, M <= MMQ_SMALL_M only: after the Mp*K*2 bytes of tiles, the same codes
 *     as int8, M rows of K bytes, each group of 8 values stored in the order
 *     (0,2,4,6,1,3,5,7): value k of token t at byte t*K + (k & ~7) +
 *     ((k & 7) >> 1) + 4*(k & 1).  The weight-streaming GEMM reads this plane.
 *     mmq_act_plane_bytes includes it in qa_bytes.
 *   M <= MMQ_FT_MAX_M only (offsets from mmq_act_ft_layout), the few-token GEMM's
 *     activation operand, with N = 16*ceil(M/16):
 *     tq (in qa, after the int8 plane if any) per k-block kb a 2*N*128-byte block
 *        at kb*2*N*128: N rows of hi then N rows of lo, row t / value k at byte
 *        t*128 + (((k/8) ^ (t%8))*16) + (k%8)*2 (f16), where for the token's
 *        super-block p = 2^(P-127), P = min(260 - E, 253) and E the f32 exponent
 *        field of the largest of its 8 chunk scales d, s = p*d (exact),
 *        s_hi = rn_f16(s), s_lo = rn_f16(s - s_hi), and for each code q:
 *        hi = rn_f16(s_hi*q), lo = rn_f16(fma(s_hi, q, -hi) + s_lo*q) (f16 fma);
 *     ip (in scales, after am) f32 1/p at index sb*MMQ_FT_MAX_M + t (t < N);
 *     fm (in scales, after ip) f32 ma = d*ssum (one f32 multiply) of chunk c of
 *        super-block sb at index (sb*8 + c % 8)*MMQ_FT_MAX_M + t (t < N).
 * -------------------------------------------------------------------------- */
#define MMQ_SMALL_M 8
#define MMQ_FT_MAX_M 64
mmq_status mmq_act_plane_bytes(int M, int K, size_t* qa_bytes, size_t* scale_bytes);
mmq_status mmq_act_scale_layout(int M, int K, size_t* pair_offset, size_t* pair_bytes,
                                size_t* am_offset, size_t* am_bytes);
/* Offsets and sizes of the few-token planes (all six 0 when M > MMQ_FT_MAX_M). */
mmq_status mmq_act_ft_layout(int M, int K, size_t* tq_offset, size_t* tq_bytes,
                             size_t* ip_offset, size_t* ip_bytes, size_t* fm_offset, size_t* fm_bytes);

/* Quantize x [M][ldx] f32 (row-major, first K values of each row used) per
 * 32-value chunk: d = amax/127 (IEEE f32 division), q = round(x/d) (IEEE f32
 * division, ties away from zero, clamped to [-127,127]; d == 0 gives q = 0),
 * ssum = sum q.  Writes qa and scales in the layout above.  x must be finite. */
mmq_status mmq_quantize_act(const float* x, int M, int K, int ldx,
                            void* qa, void* scales, mmq_stream_t s);

/* --------------------------------------------------------------------------
 * Registration-time weight repack ([r56] §2.2-§2.3 W_dsc plane: exact f16->f32
 * and int->f32 conversions, one f32 multiply, no FMA contraction; chunk-major
 * so one tile's window is contiguous; [r58] §5 names the same plane for q4_K;
 * [r56] §1 and [r58] §3.2: codes unpacked once at registration).
 *
 * For q6_K the pack calls then read FLAG word 0 back to the host and return only
 * when the stream has finished the pack (not while the stream is being captured
 * into a graph); the GEMM calls on that buffer use it to choose their kernel.  The
 * choice affects the speed only: every kernel reads FLAG itself.
 *
 * raw_blocks: od rows x id/256 super-blocks, row-major, 210 B (q6_K: ql[128]@0,
 *   qh[64]@128, int8 scales[16]@192, f16 d@208) or 144 B (q4_K: f16 d@0,
 *   f16 dmin@2, scales[12]@4 = 16 six-bit fields little-endian, fields 0..7 the
 *   scales sc_c and 8..15 the mins m_c, qs[128]@16).  Code of value e:
 *   q6_K ((ql[e/2] >> 4*(e%2)) & 15 | ((qh[e/4] >> 2*(e%4)) & 3) << 4) - 32,
 *   q4_K (qs[e/2] >> 4*(e%2)) & 15.  Value e of a q6_K block uses scales[e/16].
 *
 * packed (caller-owned, mmq_packed_weight_bytes() bytes) holds ten planes at
 * the offsets mmq_packed_weight_layout() returns; Np = 128*ceil(od/128),
 * nkb = id/64, nchunk = id/32, nsb = id/256; rows j >= od are zero:
 *   CODES  Np*id f16 integers in 16384-byte tiles (nt, kb) at (nt*nkb + kb)*16384,
 *          row r / value k at byte r*128 + (((k/8) ^ (r%8))*16) + (k%8)*2.
 *          The integer sub-block scale is folded into the code, exactly: q4_K
 *          sc_c*q (|.| <= 945); q6_K sc*q when every |scales[i]| of the tensor is
 *          <= 64 (|.| <= 2048), else sc*l with l = (q + 32) & 15 (|.| <= 1920) and
 *          the second tile in CODES2.
 *   PAIRS  Np*nchunk entries of two floats, entry (j, c) at index
 *          ((j/128)*nchunk + c)*128 + j%128:
 *            q6_K {d*scales[2*(c%8)], d*scales[2*(c%8)+1]}
 *            q4_K {d*sc_(c%8), dmin*m_(c%8)}
 *   SBD    f32 d per (row, super-block) at index ((j/128)*nsb + sb)*128 + j%128.
 *   AUX    per (row tile nt, super-block sb) an 8192-byte block at (nt*nsb + sb)*8192:
 *            q4_K: dmn = dmin*m_c split exactly into tf32 hi + lo; the hi tile then
 *                  the lo tile, row r / chunk k at (r/8)*256 + (k/4)*128 + (r%8)*16 + (k%4)*4;
 *            q6_K: the 16 scales as f32, scale s of row r at byte (s*128 + r)*4
 *                  (kept for read-back; no kernel reads it).
 *   FLAG   q6_K: uint32 word 0 = 1 if CODES are folded, word 1 = max |scales[i]|.
 *   RAW    the raw blocks re-laid for the weight-streaming GEMM, od rows x nsb
 *          blocks, row-major: q4_K 144 B [qs[128] | d | dmin | scales[12]],
 *          q6_K 224 B [ql[128] | qh[64] | scales[16] | d | 14 zero bytes].
 *   CW     compact codes for the few-token GEMM, which widens them to f16 in
 *          tensor memory: per (nt, kb) W = 2 (q4_K) or 4 (q6_K) words of 16 bytes
 *          per row, word-major: word w of row r at ((nt*nkb + kb)*W + w)*2048 + r*16.
 *          q4_K: word w holds chunk 2*kb + w, the 4-bit code of value 8u + 2p + h
 *          of the chunk (u, p = 0..3, h = 0,1) at bit 4p + 16h of its 32-bit word u.
 *          q6_K: word w holds the 16 values of sub-block w of the k-block, one byte
 *          4*(q + 32) each, value 4u + o (u, o = 0..3) at byte 2*(o & 1) + (o >> 1)
 *          of its 32-bit word u.
 *   SC     sub-block scales per (nt, sb): 16 bytes per row at ((nt*nsb + sb)*128 + r)*16:
 *          q4_K the six-bit sc_0..sc_7 then m_0..m_7, one per byte; q6_K scales[16].
 *   DM     q4_K: f32 dmin per (row, super-block) at index ((j/128)*nsb + sb)*128 + j%128
 *          (the few-token GEMM's min-term factor); q6_K: empty.
 *   CODES2 q6_K: Np*id f16 values in the CODES tile layout, 16*sc*(h - 2) with
 *          h = (q + 32) >> 4 (a multiple of 16 of magnitude <= 4096, exact) when
 *          CODES holds sc*l, so that CODES + CODES2 = sc*q; zero when CODES is
 *          folded; q4_K: empty.
 * -------------------------------------------------------------------------- */
typedef enum {
    MMQ_PLANE_CODES = 0,
    MMQ_PLANE_PAIRS = 1,
    MMQ_PLANE_SBD = 2,
    MMQ_PLANE_AUX = 3,
    MMQ_PLANE_FLAG = 4,
    MMQ_PLANE_RAW = 5,
    MMQ_PLANE_CW = 6,
    MMQ_PLANE_SC = 7,
    MMQ_PLANE_DM = 8,
    MMQ_PLANE_CODES2 = 9,
    MMQ_NUM_WEIGHT_PLANES = 10
} mmq_weight_plane;

mmq_status mmq_packed_weight_bytes(mmq_type t, int od, int id, size_t* bytes);
mmq_status mmq_packed_weight_layout(mmq_type t, int od, int id, size_t offsets[MMQ_NUM_WEIGHT_PLANES],
                                    size_t sizes[MMQ_NUM_WEIGHT_PLANES]);
mmq_status mmq_pack_weights(mmq_type t, const void* raw_blocks, int od, int id,
                            void* packed, mmq_stream_t s);

/* Fused registration of two weights that read the same input ([r58] §5, the fused
 * FFN gate/up GEMM): packs raw_a (od_a rows) and raw_b (od_b rows), both of type t
 * and width id, as ONE weight of od = od_a + od_b rows in the layout above, rows
 * [0, od_a) from raw_a and [od_a, od) from raw_b; the planes equal those of
 * mmq_pack_weights on the two raw buffers concatenated row-wise, without that copy.
 * One GEMM on it (mmq_gemm_* with od = od_a + od_b) over one set of activation
 * planes writes both outputs side by side: Y[t][j] for j < od_a is row j of a,
 * Y[t][od_a + j] row j of b.  packed must hold mmq_packed_weight_bytes(t, od, id).
 * MMQ_ERR_SHAPE for od_a or od_b < 1 or a sum over MMQ_MAX_OD; otherwise as
 * mmq_pack_weights. */
mmq_status mmq_pack_weights_fused(mmq_type t, const void* raw_a, int od_a, const void* raw_b, int od_b, int id,
                                  void* packed, mmq_stream_t s);

/* GGUF interop (registration time): nblocks q4_K (144 B) or q6_K (210 B) blocks in
 * the public ggml (llama.cpp) block layout, rewritten into the layout documented
 * above for raw_blocks, so that mmq_pack_weights can take weights read from a GGUF
 * file.  The byte offsets of d, dmin, scales and the code arrays are the same in
 * both; what moves is the position of each code and the q4_K scale packing:
 *   ggml q4_K: value 64j+l (l < 32) = low nibble of qs[32j+l], value 64j+32+l = its
 *     high nibble; sub-block s < 4: sc = S[s] & 63, m = S[s+4] & 63; s >= 4:
 *     sc = (S[s+4] & 15) | (S[s-4] >> 6) << 4, m = (S[s+4] >> 4) | (S[s] >> 6) << 4
 *     (S = scales[12]);
 *   ggml q6_K: value 128n+32p+l: low 4 bits = nibble p/2 of ql[64n+32(p%2)+l],
 *     high 2 bits = bits 2p..2p+1 of qh[32n+l]; scales[16] and d unchanged.
 * src and dst are device pointers (any alignment); dst == src converts in place;
 * other overlaps are undefined.  nblocks = 0 is a no-op.  MMQ_ERR_ARG for a bad
 * type or a null pointer. */
mmq_status mmq_convert_ggml_blocks(mmq_type t, const void* src, size_t nblocks, void* dst, mmq_stream_t s);

/* --------------------------------------------------------------------------
 * The GEMM: Y[t][j] (t < M, j < od, row stride ldy floats) is overwritten with
 * the formula at the top of this file.  packed comes from mmq_pack_weights of
 * the same (type, od, id); qa/scales from mmq_quantize_act with K = id and the
 * same M.  Four kernels compute it (mmq_last_path names the one launched;
 * mmq_debug_select_large_m_kernel can force a choice):
 *  - M <= MMQ_SMALL_M (decode and tail shapes), the weight-streaming kernel,
 *    except where the few-token kernel below is faster (measured crossovers,
 *    w = od*id: q4_K with w >= 2^24 and M >= 7, or w >= 2^25 and M >= 5; q6_K
 *    with w >= 2^25 and M >= 4): the
 *    RAW plane and the int8 activation plane, exact integer dots on the CUDA
 *    cores (dp4a), and the scales applied per chunk in the formula's own order
 *    (q4_K: Y += d_a*(d*sc_c*I) - (d_a*ssum)*(dmin*m_c); q6_K: Y +=
 *    d_a*(d*sc0*I_0 + d*sc1*I_1)), with a fixed reduction order;
 *  - otherwise for M <= MMQ_FT_MAX_M, the few-token kernel: the CW codes are
 *    widened to exact f16 integers (q4_K sc*q; q6_K sc*q when FLAG says every
 *    |scales[i]| <= 64, else the two exact tiles sc*l/4 and 4*sc*(h-2), l and h
 *    the low 4 and high 2 bits of q + 32) in tensor memory and contracted on
 *    tcgen05 against the tq operand (f16 hi and lo of p*d_a*q_a as one 2N-row
 *    operand), one f32 accumulator per stage, then d and 1/p applied per
 *    super-block; the q4_K min term sum_c (dmin*m_c)*(d_a*ssum) from DM, SC and
 *    fm in f32 FMAs (each token's sum over c = 0..7 in order); when the weight
 *    tiles are few, each is split along K over a
 *    cluster of up to 8 CTAs whose partial sums are added in rank order
 *    (deterministic);
 *  - larger M, the super-block kernel or the chunk kernel below, whichever a
 *    round-count cost model of both, fitted to GB300 timings, expects to finish
 *    first (mmq_debug_route gives the choice; q6_K whose registration found the
 *    codes in two tiles always takes the chunk kernel).  The super-block kernel:
 *    the activation operand p*d_a*q_a as an f16 hi + lo pair
 *    (about 2^-21 relative per value) times the exact f16 CODES (and CODES2 for
 *    two-tile q6_K, a second pair of MMAs into the same accumulator), summed over
 *    a whole super-block in f32, then d and 1/p per super-block.  In both tile
 *    kernels, when the last round of tiles fills at most half the SMs (or all
 *    tiles do), those tiles run as two K-halves added into Y after a zeroing
 *    kernel, 0 + a + b, the same in either order;
 *  - the chunk kernel: the integer dots sum_chunk (sc*q)*q_a run
 *    exactly (codes held as f16 integers, two-tile q6_K as two MMAs per 16
 *    values, every partial sum an integer below 2^24 in the f32 accumulator)
 *    and the f32 scales are applied per chunk (d_a) and per super-block (d).
 * The super-block and chunk kernels compute the q4_K min term sum_c
 * (d_a*ssum)*(dmin*m_c) as a tf32 hi/lo tensor-core contraction (relative error
 * about 2^-21 per product), each TMEM accumulator covering at most 64
 * super-blocks before it is added into Y's f32 sums.
 * Y is deterministic for given inputs and kernel.  Rows t >= M and columns
 * j >= od are never written.  ldy >= od.
 * -------------------------------------------------------------------------- */
mmq_status mmq_gemm_q6k(const void* packed, int od, int id, const void* qa, const void* scales,
                        int M, float* Y, int ldy, mmq_stream_t s);
mmq_status mmq_gemm_q4k(const void* packed, int od, int id, const void* qa, const void* scales,
                        int M, float* Y, int ldy, mmq_stream_t s);

/* Debug/verification: the same GEMM kernel (same staging, same tensor-core
 * contraction) writes the raw integer dots it accumulates instead of Y, as f32
 * values holding the exact integers, at dots[(t*od + j)*nsub + s]:
 *   q4_K: nsub = id/32, s = chunk c: sc_c * sum(q * q_a)
 *   q6_K: nsub = id/32, s = chunk c: sc0*I_0 + sc1*I_1
 * (I_h = sum(q * q_a) over the chunk's 16-value half h; |value| < 2^24). */
mmq_status mmq_debug_gemm_dots(mmq_type t, const void* packed, int od, int id, const void* qa,
                               const void* scales, int M, float* dots, mmq_stream_t s);

/* Debug/verification, host logic only (no CUDA call): the kernel the default
 * selection of mmq_gemm_* gives for (t, od, id, M) on a device with nsm SMs, for
 * q6_K codes folded (fold = 1), in two tiles (0) or of unknown state (-1, taken as
 * folded; q4_K ignores fold): *kernel = 0 weight-streaming, 1 chunk, 2 super-block,
 * 3 few-token.  MMQ_ERR_ARG for a null kernel, nsm < 1 or fold outside -1..1;
 * otherwise the shape errors of the GEMM calls. */
mmq_status mmq_debug_route(mmq_type t, int od, int id, int M, int fold, int nsm, int* kernel);

/* Debug/verification: which kernel computes Y (process-wide).
 *   0 (default): as described above the GEMM calls;
 *   1: the chunk kernel for every M > MMQ_SMALL_M (128-token tiles);
 *   2: the super-block kernel for every M > MMQ_SMALL_M;
 *   3: as 0, but the few-token kernel never splits a tile over a CTA cluster;
 *   4: as 0, but the few-token kernel also for M <= MMQ_SMALL_M.
 * Returns MMQ_ERR_ARG for any other value.  Not thread-safe against GEMM calls
 * in flight on other host threads. */
mmq_status mmq_debug_select_large_m_kernel(int which);

/* Debug/verification of the timeout path (a loud error, never a silent wrong
 * result: [r56] §3.1).  Arms a one-shot injection for the next GEMM launch that
 * runs a tile kernel (M > MMQ_SMALL_M), or attention launch whose CTAs form no
 * clusters: its waits give up after limit_ns (1 us .. 2 s) instead of about two
 * seconds, and the producer of its first CTA leaves operand fill number `fill` out
 * (0-based, counted over that CTA's k-blocks; over the K and V halves of a prompt's
 * pairs of pages, for its first rows of kv head 0; a few rows' attention leaves its first
 * page out whatever `fill` is), so the wait for it runs out, the launch exits early and
 * mmq_get_device_error() then returns MMQ_ERR_TIMEOUT (and clears the word).
 * That launch takes no CTA-cluster split.  Its result is undefined.  fill < 0
 * disarms a pending injection.  MMQ_ERR_ARG for a limit outside the range.
 * Process-wide host state; no CUDA call. */
mmq_status mmq_debug_inject_wait_timeout(int fill, unsigned long long limit_ns);

/* --------------------------------------------------------------------------
 * A 4-bit key/value cache and attention over it.
 *
 * The cache is a pool of pages of MMQ_KV_PAGE tokens.  A page holds one piece of
 * 72 * head_dim bytes per kv head (mmq_kv_page_bytes for all heads), page p at
 * pages + p * kv_heads * 72 * head_dim, head h's piece h pieces further on.  Groups of
 * 32 consecutive values of one head of one token share a scale s of 7 significant
 * bits in [2^-14, 896], held as f16; code n = 0..15 stands for s * (n - 8) (exact in
 * f16).  4.5 bits a value in all.  Inside a piece, D = head_dim, NG = D/32 groups:
 *   K codes   at 0: token t (0..63), group g: the 16-byte chunk at t*(D/2) +
 *             16*(g ^ ((t >> 1) & 3)) for D = 128, 16*(g ^ ((t >> 2) & 1)) for D = 64;
 *             the code of value 8u + 2p + h of the group (u, p = 0..3, h = 0, 1) at bit
 *             4p + 16h of the chunk's 32-bit word u.
 *   K scales  at 32 D: f16 [t][g].
 *   V codes   at 36 D: pair p = t/2, block a = value/16: the 16-byte chunk at p*D +
 *             16*(a ^ turn), turn = ((p >> 2) ^ (2p & 6)) & 7 for D = 128,
 *             ((p >> 2) ^ (p & 2)) & 3 for D = 64; the code of value 16a + 4u + i
 *             (u, i = 0..3) of token 2p + e at bit 4i + 16e of the chunk's word u.
 *   V scales  at 68 D: f16 [p][g][e].
 * Slots that no token was written to may hold anything.
 *
 * A batch of sequences: table[b * max_pages + i] is the page of positions 64 i ..
 * 64 i + 63 of sequence b, length[b] its token count.  The calls work on packed rows of
 * new tokens: rows start[b] <= r < start[b + 1] (start has batch + 1 entries,
 * start[0] = 0 and start[batch] = ntok) are the last tokens of sequence b, row r at
 * position length[b] - start[b + 1] + r.  table, start and length are read on the
 * device.  A page id outside [0, num_pages) or a position outside [0, 64 max_pages) is
 * not followed: such a token is not written and reads as zeros, such keys are not
 * there for the attention, and mmq_get_device_error then returns MMQ_ERR_ARG.  So it does
 * for packed rows outside start[0] .. start[batch], or of a sequence whose start leads outside
 * [0, ntok]: they are not written, read as zeros, and are zeros as results of the attention.
 * -------------------------------------------------------------------------- */
#define MMQ_KV_PAGE 64
#define MMQ_KV_MAX_HEADS 1024
#define MMQ_KV_MAX_BATCH (1 << 20)
#define MMQ_KV_MAX_PAGES (1 << 24)

typedef enum { MMQ_F32 = 0, MMQ_F16 = 1, MMQ_BF16 = 2 } mmq_dtype;

typedef struct {
    void* pages;              /* device, 16-byte aligned */
    const int32_t* table;     /* device, batch * max_pages */
    const int32_t* start;     /* device, batch + 1 */
    const int32_t* length;    /* device, batch */
    int num_pages;
    int kv_heads;             /* 1 .. MMQ_KV_MAX_HEADS */
    int head_dim;             /* 64 or 128 */
    int batch;                /* 1 .. MMQ_KV_MAX_BATCH */
    int max_pages;            /* 1 .. MMQ_KV_MAX_PAGES */
} mmq_kv_cache;

/* Rows [token][head][head_dim] of a tensor; strides in elements, >= 0, the last
 * dimension contiguous.  Any alignment of an element; rows aligned to four elements are
 * moved four at a time.  Rows that a call writes may not overlap (MMQ_ERR_ARG). */
typedef struct {
    void* data;
    int dtype;                /* mmq_dtype */
    long long token_stride;
    long long head_stride;
} mmq_rows;

/* Bytes of one page. */
mmq_status mmq_kv_page_bytes(int kv_heads, int head_dim, size_t* bytes);

/* Quantise k and v (one dtype, ntok rows of kv_heads heads) into the cache.  Per group:
 * s = amax / 7.5 (IEEE f32 division) rounded up to 7 significant bits and limited to
 * [2^-14, 896]; n = rint(x / s) (IEEE f32 division, ties to even) limited to -8..7,
 * plus 8.  Magnitudes over 6720 saturate; NaN is stored as 0.  Tokens of one call must
 * have places of their own.  ntok = 0 is a no-op. */
mmq_status mmq_kv_write(const mmq_kv_cache* c, const mmq_rows* k, const mmq_rows* v, int ntok, mmq_stream_t s);

/* The reverse: rows of k and v get the values that the cache holds for those tokens
 * (exact in f32 and f16, rounded to nearest in bf16).  With start[b + 1] - start[b] =
 * length[b] whole sequences are read. */
mmq_status mmq_kv_read(const mmq_kv_cache* c, const mmq_rows* k, const mmq_rows* v, int ntok, mmq_stream_t s);

/* Attention of the new tokens' queries over the cache (their own keys included: write
 * them first):
 *   out[r][h] = sum_j w_j v_j / sum_j w_j,   w_j = exp(scale * q[r][h] . k_j),
 * j over the keys that a query at position p sees: j <= p, and with window > 0 also
 * j > p - window or j < sinks (the first tokens that stay visible).  Head h reads kv
 * head h / (heads / kv_heads).  A row that sees no key is 0.  q and out have one dtype;
 * sums, the softmax and both products' accumulators are f32.  For f32 rows the queries
 * and the weights enter the products as pairs of f16 (22 bits, a weight no finer than 2^-38 of
 * the row's largest).  The tensor cores cut their sums toward zero, by up to 2^-23 at each
 * product; f32 rows add up at most 160 products before they move such a sum to one that is
 * rounded.  For values of one sign that is below 1e-5 of the result where no key outweighs
 * the others (2.3e-6 on a prompt of 3314 tokens, where f32 arithmetic loses 1.0e-6) and up to
 * 2.5e-5 where one outweighs a long tail.  For 16-bit rows the weights are rounded to f16 and no
 * finer than 2^-32 of the row's largest.  Such errors are relative to the largest values that
 * have weight: where the key that outweighs the others has a value near zero, they are more of
 * the result.  q must be finite: a row that is not has no number for a result and touches no
 * other row.
 * scale > 0, a normal number up to 1e38.
 *   max_q   at least the largest start[b + 1] - start[b] (else rows past it may be left
 *           out as zeros, and mmq_get_device_error then returns MMQ_ERR_ARG)
 *   max_kv  about the largest length[b]; it guides how the work is cut, any value is right
 *           (one past 64 * max_pages counts as that; one far too low costs time and, for
 *           16-bit rows, digits, as their sums over the keys past it stay whole: f16 rows
 *           lose 4.3e-4 of values of one sign over 65536 such keys)
 * The work is cut into parts whose sums meet in the workspace (of
 * mmq_kv_attend_workspace_bytes for the same arguments, 16-byte aligned; may be NULL when
 * that is 0) in a fixed order, so results do not vary from call to call.  out may not
 * overlap q, the cache or the workspace. */
mmq_status mmq_kv_attend_workspace_bytes(const mmq_kv_cache* c, int dtype, int heads, int ntok, int max_q, int max_kv,
                                         int window, int sinks, size_t* bytes);
mmq_status mmq_kv_attend(const mmq_kv_cache* c, const mmq_rows* q, const mmq_rows* out, int heads, int ntok, int max_q,
                         int max_kv, float scale, int window, int sinks, void* workspace, size_t workspace_bytes,
                         mmq_stream_t s);

/* --------------------------------------------------------------------------
 * A cache held to a budget of tokens.
 *
 * weights: f32 [num_pages][kv_heads][MMQ_KV_PAGE], what each cached token's key of each kv head
 * has received of the softmax so far, beside the pages of the cache (16-byte aligned).
 * -------------------------------------------------------------------------- */

/* mmq_kv_attend (same arguments, same result), and the weight that each key received, added to
 * what it had: for kv head h and every token j of every sequence with new tokens,
 *   new_weights[h][j] = (j < length - new ? decay * weights[h][j] : 0) + sum over the sequence's new
 *   rows and the heads that read h of w_j / sum_i w_i
 * (w as above; 0 for keys that a row does not see; new = start[b + 1] - start[b], whose tokens start
 * from 0, so nothing has to be cleared).  decay in [0, 1].  new_weights may be weights; a buffer of
 * its own keeps the old ones, for a step that may be taken back.  Slots past the last token, and
 * pages of no sequence with new tokens, are left as they were.  A row that is not finite, or past
 * max_q (see there), adds nothing.  The sums are f32, in a fixed order: the same call gives the same bits.
 * No two sequences of a call that have new tokens may share a page (a prefix, say): what its weights then
 * are is not defined and varies from call to call (one's sum, or, in place, one added to the other with
 * the decay applied twice), and nothing reports it.  A call for each of them is defined: each adds to
 * what the one before left.
 * Tokens that came in by another call (mmq_kv_attend) hold what the memory held; clear that first.
 * Workspace: mmq_kv_attend_weights_workspace_bytes, more than 0 where ntok is, and what it holds before
 * does not matter.  Up to 16 to 48 rows (new tokens times the heads that read a kv head, by type and
 * head_dim) it has room for the scores of max_kv keys, up to a gigabyte, so that K is read once.  Above
 * 128 rows it has the rows of all heads in 16 bits, twice that for f32 ones, and up to 8 more rows of
 * each kv head for each sequence that may have new tokens.
 * max_kv: with scores kept, keys past it are computed again value by value, and at once cost much more than
 * their reading (one token on 131071 keys, 32 heads on 8: 56 us; with max_kv 130000 0.27 ms, with 65536 1.2 ms,
 * with 1 41 ms).  Where lengths grow while a captured call is replayed, give the length they may reach. */
mmq_status mmq_kv_attend_weights_workspace_bytes(const mmq_kv_cache* c, int dtype, int heads, int ntok, int max_q,
                                                 int max_kv, int window, int sinks, size_t* bytes);
mmq_status mmq_kv_attend_weights(const mmq_kv_cache* c, const mmq_rows* q, const mmq_rows* out, int heads, int ntok,
                                 int max_q, int max_kv, float scale, int window, int sinks, const float* weights,
                                 float* new_weights, float decay, void* workspace, size_t workspace_bytes,
                                 mmq_stream_t s);

/* Eviction: of each sequence min(length, keep) tokens go to the pages of new_table ([batch][new_pages]
 * page ids, new_pages * MMQ_KV_PAGE >= keep), in their order, with their weights.  Where length >
 * keep those are, per kv head, the first `first` tokens, the last `last` (first + last <= keep), and the
 * keep - first - last of the rest with the largest weights; of equal ones the earlier stays, and a
 * weight that is no number counts as the least.  So a slot may hold different tokens in different
 * heads.  Codes and scales are moved, not computed anew.
 *   new_length  [batch]: min(length, keep); may be c->length
 *   kept        [batch][kv_heads][keep]: the old place of the token in each new one, -1 past new_length
 *   max_kv      about the longest length, as for mmq_kv_attend
 * c->start is not read.  The old pages are only read, so other sequences may share them (for their
 * weights see mmq_kv_attend_weights); the new ones may not be among them or be named twice (what they
 * then hold is undefined).  Slots past new_length are left as they were.  A token whose old page is no page of the pool counts as the
 * least weight and moves as zeros, one whose new page is none does not move, and mmq_get_device_error
 * then returns MMQ_ERR_ARG.
 * A window of mmq_kv_attend counts slots: after an eviction it reaches further back than before.
 * Keys keep the rotation they were written with; new ones go on with the positions of the text. */
mmq_status mmq_kv_evict(const mmq_kv_cache* c, float* weights, const int32_t* new_table, int new_pages, int keep,
                        int first, int last, int max_kv, int32_t* new_length, int32_t* kept, mmq_stream_t s);

/* --------------------------------------------------------------------------
 * Rotary positions.  With f_i the angle per position of pair i, the values (a, b) of the pair in a
 * row at position p become (a c - b s, a s + b c), c = m cos(p f_i), s = m sin(p f_i).  Pair i is values
 * i and i + rot_dim / 2 of the head, or 2 i and 2 i + 1 interleaved; values from rot_dim on stay.
 * cos and sin are f32 numbers next to the true ones however far the position; products and sums are
 * f32, rounded one by one, and the result is rounded once to the rows' type.
 * -------------------------------------------------------------------------- */
#define MMQ_ROPE_MAX_DIM 1024

typedef struct {
    const uint64_t* turns;    /* device, rot_dim / 2, 8-byte aligned: f_i / (2 pi) * 2^64 modulo 2^64 */
    int rot_dim;              /* even, 2 .. head_dim */
    int interleaved;          /* 0 or 1 */
    float magnitude;          /* m, finite; 1 where nothing asks for another */
} mmq_rope_plan;

typedef enum {
    MMQ_ROPE_PLAIN = 0,       /* f_i = base^(-2 i / rot_dim) */
    MMQ_ROPE_LINEAR = 1,      /* f_i / factor: positions interpolated */
    MMQ_ROPE_NTK = 2,         /* base * factor^(rot_dim / (rot_dim - 2)) for base: the slowest pair is
                                 factor times slower, the fastest as it was */
    MMQ_ROPE_YARN = 3,        /* (1 - r_i) f_i + r_i f_i / factor, r_i = (i - lo) / (hi - lo) within [0, 1], lo
                                 and hi the (real) pairs, rounded down and up, that make 32 turns and 1
                                 turn over `original` positions; magnitude 0.1 ln(factor) + 1 (B. Peng et
                                 al., YaRN, 2023) */
    MMQ_ROPE_BANDS = 4        /* n_i f_i + (1 - n_i) f_i / factor, n_i = (t_i - 1) / 3 within [0, 1], t_i the
                                 turns of the pair over `original` positions */
} mmq_rope_scaling;

/* Host only: the f_i (freq, rot_dim / 2 doubles) and the magnitude of a scaling.  base > 1, factor >= 1
 * (not looked at by PLAIN), original >= 1 (looked at by YARN and BANDS). */
mmq_status mmq_rope_frequencies(mmq_rope_scaling scaling, int rot_dim, double base, double factor, double original,
                                double* freq, float* magnitude);
/* Host only: the turns of n frequencies (magnitudes up to 1e6), to copy to the device. */
mmq_status mmq_rope_turns(const double* freq, int n, uint64_t* turns);

/* out = x turned, rows of `heads` heads of head_dim values (up to MMQ_ROPE_MAX_DIM) of one dtype, row r
 * at position pos[r] (device, any int32).  out may be x (same data and strides); other overlaps are
 * undefined.  A value that is not finite touches its pair alone. */
mmq_status mmq_rope(const mmq_rope_plan* p, const mmq_rows* x, const mmq_rows* out, const int32_t* pos, int heads,
                    int head_dim, int ntok, mmq_stream_t s);

/* mmq_rope of q into q_out (which may be q), and mmq_kv_write of k, turned, and v, in one launch.  All
 * rows have one dtype; the turned k is quantised as it is in f32, not rounded to that type before.  pos
 * is the rotation's position and need not be the place in the cache (after an eviction it is not). */
mmq_status mmq_kv_write_rope(const mmq_kv_cache* c, const mmq_rope_plan* p, const mmq_rows* q, const mmq_rows* q_out,
                             int heads, const mmq_rows* k, const mmq_rows* v, const int32_t* pos, int ntok,
                             mmq_stream_t s);

/* Synchronizes `s`, then reports and clears the sticky device error words:
 * MMQ_ERR_TIMEOUT if a bounded wait expired since the last call, else MMQ_ERR_ARG if a
 * cache call met a page, a position or a row count outside what it was given,
 * MMQ_ERR_CUDA if the synchronization failed, else MMQ_OK. */
mmq_status mmq_get_device_error(mmq_stream_t s);

const char* mmq_status_string(mmq_status st);

/* Label of the path the most recent GEMM launch took (liveness check,
 * [r56] §3.2 and §4: a fast path needs a visible label because parity alone
 * cannot show it ran). */
const char* mmq_last_path(void);

/* Number of kernel launches the library has made in this process (every entry
 * point that launches adds the kernels it launched: prepass 1, repack 4 or 5,
 * GEMM 1, or 2 when K-half tiles are first zeroed; cache write and read 1, attention 1,
 * or 2 when parts are joined through the workspace, and for the weights 1 more, or 2 when a
 * sequence's kv head has more than 128 rows; eviction 2; rotary positions 1, with the cache write or
 * without). */
unsigned long long mmq_launch_count(void);

/* Library version string. */
const char* mmq_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MMQ_GB300_H */
