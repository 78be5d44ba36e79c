/*
 * splitzip.h -- C ABI of libsplitzip, a lossless exponent codec for BF16 and
 * FP8 E5M2 KV-cache tensors on AMD Instinct MI355X (gfx950).
 *
 * The method is SplitZip ("SplitZip: Ultra Fast Lossless KV Compression for
 * Disaggregated LLM Serving", arXiv 2605.01708v2).  Its pages state the
 * problem this ABI serves: KV tensors must reach the decode side bit for bit,
 * and the codec must plug into a serving stack without touching model
 * execution (authors' abstract; Spanish technical summary, "Metodologia").
 *
 * Conventions for every call:
 *   - extern "C", never throws, returns an int status (SPLITZIP_OK = 0 or a
 *     negative SPLITZIP_E_* code); sizes are element or byte counts.
 *   - "d_" pointers are device memory (hipMalloc'd, or any memory the GPU
 *     can address); "h_" pointers are host memory.  The caller owns every
 *     buffer.  No call allocates device or host memory (the pipelined
 *     transfer creates HIP events for the duration of its call).
 *   - GPU work is enqueued on `stream` (NULL = the default stream) and is not
 *     waited for.  Host-detectable argument errors return at once and enqueue
 *     nothing.  A failed kernel launch returns SPLITZIP_E_HIP.
 *   - Calls on different streams may run concurrently when their buffers are
 *     disjoint; the library keeps no mutable global state, except the device
 *     array behind splitzip_compress_static (whose calls must not overlap on
 *     one GPU; see there).
 *   - The device calls (compress, decompress and their variants, the device
 *     calibration) only launch kernels on `stream`: no allocation, memset or
 *     synchronization, so they can be captured in a HIP graph and replayed.
 *     Decompress takes in_bytes as an upper bound (the buffer's size), so a
 *     captured decompress serves streams of any size S <= in_bytes.
 *
 * Stream format "SZ1" (little-endian; A(x) = x rounded up to a multiple of
 * 256; n elements, C = ceil(n / 65536) chunks, K codebooks, E escapes):
 *   0    u32 magic 0x00315A53        4  u16 version 1
 *   6    u8  dtype                    7  u8  log2 chunk size = 16
 *   8    u64 n                        16 u64 E
 *   24   u64 total stream bytes S     32 u32 C      36 u32 K
 *   40   u64 elements per segment (n when K == 1)
 *   48   16 zero bytes
 *   64          K codebooks of 16 bytes (byte k = exponent of 4-bit code k)
 *   64 + 16K    C + 1 u64: escapes before chunk c (off[C] = E)
 *   N0 = A(64 + 16K + 8(C + 1)): 4-bit codes, two per byte, even element in
 *        the low nibble; an escaped element has code 0        (ceil(n/2) B)
 *   N1 = N0 + A(ceil(n/2)): sign|mantissa
 *        BF16: one byte per element, sign at bit 7, mantissa bits 6..0 (n B)
 *        E5M2: 3 bits per element (sign << 2 | mantissa), 8 elements per 3
 *              little-endian bytes, element j of a group at bits 3j  (3 ceil(n/8) B)
 *   P  = N1 + A(sign|mantissa bytes): E escape records of 3 bytes
 *        [position in chunk, low byte][high byte][raw exponent], in element order
 *   S  = P + 3E.  All bytes between sections are zero.
 * Chunk c is coded with codebook 0 when K == 1, else with codebook
 * floor(65536 c / segment_elems).
 */
#ifndef SPLITZIP_H
#define SPLITZIP_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Element types.  BF16: 1 sign, 8 exponent, 7 mantissa bits (English
 * explainer, "1. The 'Note' Structure").  FP8 E5M2: 1 sign, 5 exponent,
 * 2 mantissa bits (technical summary, "Contribuciones Clave" 4). */
typedef enum { SPLITZIP_BF16 = 1, SPLITZIP_FP8_E5M2 = 2 } splitzip_dtype;

enum {
  SPLITZIP_OK = 0,
  SPLITZIP_E_INVALID = -1,  /* bad argument: null/misaligned pointer, dtype, sizes, segments */
  SPLITZIP_E_CAPACITY = -2, /* output buffer smaller than splitzip_max_compressed_size() */
  SPLITZIP_E_CODEBOOK = -3, /* codebook entries repeated or out of range for the dtype */
  SPLITZIP_E_CORRUPT = -4,  /* stream fails validation (reported through d_status) */
  SPLITZIP_E_HIP = -5,      /* a HIP launch failed */
  SPLITZIP_E_TOO_LARGE = -6, /* input beyond splitzip_compress_static's limit */
  SPLITZIP_E_NONFINITE = -7 /* a NaN or infinity met by splitzip_kv4_append (reported through d_status) */
};

/* Offline calibration (technical summary, "Metodologia / Codificacion de
 * Longitud Fija" and "Optimizacion"; "Resultados / Calibracion"; abstract):
 * histogram the exponents of n_elems host samples and return the 16 most
 * frequent exponent values in codebook_out[0..15], most frequent first;
 * equal counts go to the lower exponent; values never seen fill the
 * remaining slots in ascending order, so the 16 entries are always distinct.
 * host_samples: n_elems BF16 (uint16 bit patterns) or E5M2 (uint8) values in
 * host memory; may be NULL only when n_elems == 0.  Synchronous, host only.
 * Returns SPLITZIP_OK or SPLITZIP_E_INVALID. */
int splitzip_calibrate(int dtype, const void* host_samples, size_t n_elems, uint8_t codebook_out[16]);

/* Bytes the caller must provide as d_out of splitzip_compress for n_elems
 * elements and n_codebooks codebooks: the largest possible stream (every
 * element escaped) rounded up to 256, plus the encoder's workspace: per
 * 8192-element tile 2052 bytes (a count and a staging slot for up to 512
 * escape records), per 64 tiles 8 bytes and per 4096 tiles 8 bytes, with
 * 256-byte alignment.  Returns 0 for an invalid dtype,
 * n_codebooks == 0 or n_elems > 2^36 (the largest n any call accepts: every
 * kernel grid then stays below 2^32 work-items; 2^36 BF16 elements are
 * 128 GiB). */
size_t splitzip_max_compressed_size(int dtype, size_t n_elems, uint32_t n_codebooks);

/* Encode (technical summary, "Estrategia de Codificacion"; abstract; English
 * explainer, "3. The SplitZip Strategy"): split every element into exponent
 * and sign|mantissa, map the exponent through its chunk's codebook to a 4-bit
 * code, and route exponents outside the codebook to the escape records.
 *   d_in          n_elems elements (BF16 as uint16, E5M2 as uint8), 16-byte aligned.
 *   h_codebooks   n_codebooks x 16 bytes, host memory, read before return.
 *   segment_elems elements per codebook; ignored when n_codebooks == 1,
 *                 else a non-zero multiple of 65536 with
 *                 n_codebooks * segment_elems >= n_elems.
 *   d_out         out_capacity bytes, 16-byte aligned; the stream is written
 *                 at its start; bytes after the stream are the encoder's
 *                 workspace and are overwritten.
 *   d_out_bytes   optional (may be NULL): receives the stream size S, written
 *                 by the GPU when the encode completes (device or pinned host
 *                 memory, 8-byte aligned).
 * The stream is byte-for-byte deterministic for given inputs.  d_in is not
 * modified.  Returns SPLITZIP_OK, SPLITZIP_E_INVALID, SPLITZIP_E_CODEBOOK,
 * SPLITZIP_E_CAPACITY or SPLITZIP_E_HIP. */
int splitzip_compress(int dtype, const void* d_in, size_t n_elems, const uint8_t* h_codebooks,
                      uint32_t n_codebooks, size_t segment_elems, void* d_out, size_t out_capacity,
                      uint64_t* d_out_bytes, hipStream_t stream);

/* Decode (technical summary, "Estrategia de Decodificacion / Paralelismo"
 * and "Correccion"; English explainer, "4. Why It's Fast"): map every 4-bit
 * code through its codebook, recombine with the sign|mantissa bits, then
 * overwrite the exponent of every escaped element with its raw value.  One
 * kernel launch.
 *   d_in      the stream (in_bytes >= its size S, 16-byte aligned).
 *   dtype, n_elems must match the stream header.
 *   d_out     n_elems elements, 16-byte aligned.
 *   d_status  optional (may be NULL), device int32, sticky: the caller sets
 *             it to SPLITZIP_OK (0) beforehand; the GPU writes
 *             SPLITZIP_E_CORRUPT into it if it finds the stream invalid and
 *             never clears it, so one word can watch many calls.  d_out is
 *             then unspecified.  Invalid means: bad magic, version, dtype, n,
 *             non-zero reserved header bytes, chunk count, codebook count
 *             or segment size; E > n or
 *             S != P + 3E or S > in_bytes; any of the K codebooks (used by a
 *             chunk or not) with a repeated entry or, for E5M2, an entry of
 *             32 or more; chunk offsets not starting at 0, decreasing, above
 *             E, not ending at E, or giving a chunk more records than
 *             elements; an escape position outside its chunk or not above
 *             the previous one of the chunk; an escape value of 32 or more
 *             (E5M2).  Every stream the encoder writes passes these checks,
 *             and they are the oracle's.  Every read stays inside in_bytes.
 * Returns SPLITZIP_OK, SPLITZIP_E_INVALID or SPLITZIP_E_HIP. */
int splitzip_decompress(const void* d_in, size_t in_bytes, int dtype, size_t n_elems, void* d_out,
                        int32_t* d_status, hipStream_t stream);

/* Static text for a status code. */
const char* splitzip_status_string(int status);

/* splitzip_compress for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  The encoder's workspace (per-tile escape counts and record
 * staging slots) is the library's own device array (about 4 MiB per GPU,
 * kept until the process ends) instead of the tail of d_out.  Inputs of at
 * most 512 tiles (4M BF16 or 8M E5M2 elements) take one launch whose
 * workgroups exchange their tiles' escape counts through that array (a wait
 * for a count is bounded: SPLITZIP_STATIC_WAIT_POLLS polls, 64 if unset,
 * after which the count is computed from the input); larger ones take the
 * launches of splitzip_compress.  d_out only needs room for the largest
 * stream:
 *   out_capacity >= A(P + 3 n_elems), P as in the layout above with
 *   n_elems escapes (splitzip_max_compressed_size minus the workspace).
 * Limit: n_elems <= 2048 * 8192 (BF16) or 2048 * 16384 (E5M2), 32 MiB of
 * input, else SPLITZIP_E_TOO_LARGE.  Other arguments, errors and the stream
 * are those of splitzip_compress: the stream is byte for byte the one
 * splitzip_compress writes.  No hipMalloc, hipFree, memset or host
 * synchronization, so it can be captured in a HIP graph.  Every call on one
 * GPU shares that GPU's workspace: calls that overlap on one GPU (two
 * streams, two host threads) race and may write wrong streams; serialize
 * them.  Calls that follow a race are not affected by it.  The stream
 * passed must belong to the current device.
 * Returns SPLITZIP_OK, SPLITZIP_E_INVALID, SPLITZIP_E_CODEBOOK,
 * SPLITZIP_E_CAPACITY, SPLITZIP_E_TOO_LARGE or SPLITZIP_E_HIP. */
int splitzip_compress_static(int dtype, const void* d_in, size_t n_elems, const uint8_t* h_codebooks,
                             uint32_t n_codebooks, size_t segment_elems, void* d_out, size_t out_capacity,
                             uint64_t* d_out_bytes, hipStream_t stream);

/* ---- Ablation variants (BF16) ---------------------------------------------
 * The two designs the pages measure against the top-16 codec (technical
 * summary, "Metodologia / Decision de Diseno" and "Resultados"), as streams
 * of their own, to compare decode speed and size on this GPU:
 *   SPLITZIP_VARIANT_TOP15_SENTINEL  codebook entries 0..14 get codes 0..14;
 *     code 15 marks an escape, whose raw exponent is the next byte of the
 *     escape section (no positions: the pages' design with less side data).
 *   SPLITZIP_VARIANT_TOP8            codebook entries 0..7 get 3-bit codes,
 *     8 codes per 3 little-endian bytes (element j at bit 3j); escapes are the
 *     codec's 3-byte position records.
 * Layout: the SZ1 layout with header byte 48 = the variant, the code section
 * of ceil(n/2) (top-15) or 3 ceil(n/8) (top-8) bytes, and E escape bytes
 * (top-15) or 3E (top-8) at the end.  Codebooks are 16 distinct entries per
 * segment as for splitzip_compress; the variant uses the first 15 or 8.
 * The arguments, alignment, workspace and status conventions are those of
 * splitzip_max_compressed_size, splitzip_compress and splitzip_decompress,
 * except that the top-8 workspace stages up to 1024 escape records per
 * 8192-element tile (4 KiB per tile, against 2 KiB for the codec's 512);
 * dtype is BF16.  An invalid variant returns 0 / SPLITZIP_E_INVALID. */
typedef enum { SPLITZIP_VARIANT_TOP15_SENTINEL = 1, SPLITZIP_VARIANT_TOP8 = 2 } splitzip_variant;

size_t splitzip_variant_max_compressed_size(int variant, size_t n_elems, uint32_t n_codebooks);

int splitzip_variant_compress(int variant, const void* d_in, size_t n_elems, const uint8_t* h_codebooks,
                              uint32_t n_codebooks, size_t segment_elems, void* d_out, size_t out_capacity,
                              uint64_t* d_out_bytes, hipStream_t stream);

/* Top-8: one workgroup per 8192-element tile, as splitzip_decompress.
 * Top-15 + sentinel: one workgroup per chunk, which counts the sentinels
 * before every element to find its value (the irregular step the pages
 * attribute the design's slower decode to). */
int splitzip_variant_decompress(int variant, const void* d_in, size_t in_bytes, size_t n_elems, void* d_out,
                                int32_t* d_status, hipStream_t stream);

/* ---- On-device calibration ------------------------------------------------
 * The pages calibrate offline, so that no histogram is built on the critical
 * path (technical summary, "Optimizacion" and "Resultados / Calibracion";
 * abstract).  splitzip_calibrate_device builds that histogram on the GPU, to
 * measure what calibrating online would cost and to calibrate per tensor or
 * per layer at run time.  The codebooks equal splitzip_calibrate's on the same
 * samples: the 16 most frequent exponents, most frequent first, equal counts
 * to the lower exponent, unseen exponents filling up in ascending order.
 *
 * splitzip_calibrate_device_work_bytes: bytes of d_work for n_codebooks
 * segments (8 per histogram bin: 256 bins BF16, 32 E5M2), 0 for an invalid
 * dtype or n_codebooks outside 1..65535. */
size_t splitzip_calibrate_device_work_bytes(int dtype, uint32_t n_codebooks);

/* splitzip_calibrate_device: one codebook per segment of d_samples.
 *   d_samples       n_elems elements on the device (BF16 as uint16, E5M2 as
 *                   uint8), 16-byte aligned.
 *   segment_elems   elements per segment, ignored when n_codebooks == 1
 *                   (one segment: the whole tensor); else segment k covers
 *                   [k * segment_elems, min((k + 1) * segment_elems, n)) and
 *                   n_codebooks * segment_elems >= n_elems.  A segment with no
 *                   elements gets the codebook 0, 1, ..., 15.
 *   d_codebooks_out n_codebooks x 16 bytes, device memory, written by the GPU.
 *   d_work          work_bytes of device memory, 8-byte aligned, overwritten.
 * Stream-ordered, three launches, no host synchronization.  Returns
 * SPLITZIP_OK, SPLITZIP_E_INVALID, SPLITZIP_E_CAPACITY or SPLITZIP_E_HIP. */
int splitzip_calibrate_device(int dtype, const void* d_samples, size_t n_elems, size_t segment_elems,
                              uint32_t n_codebooks, uint8_t* d_codebooks_out, void* d_work, size_t work_bytes,
                              hipStream_t stream);

/* ---- Chunk-pipelined transfer through a host link -------------------------
 * The pages' setting is a KV cache moving from a prefill node to a decode
 * node over a 50-100 GB/s link, where the codec shrinks the transferred bytes
 * and pays for itself (technical summary, "Planteamiento del Problema" and
 * "Resultados": 1.22-1.32x faster transfers).  On one GPU the link is the
 * PCIe path to pinned host memory: each group of group_elems elements is
 * compressed (splitzip_compress), copied to host memory and back by the copy
 * engines, and decompressed (splitzip_decompress) into d_out, with up to
 * `depth` groups in flight.  A compressed group's size exists only on the
 * device: the encoder writes it into the link buffer, and the host, one group
 * behind the encoder, polls it before queuing that group's copies.
 *
 * Each group is a complete SZ1 stream of its own elements.  group_elems is a
 * non-zero multiple of 65536; with n_codebooks > 1, group_elems is a multiple
 * of segment_elems or divides it, so a group uses the codebooks of the
 * segments it covers.  depth is 2..32.
 *
 * splitzip_pipeline_sizes: bytes of the device work area (2 * depth slots)
 * and of the pinned host link buffer (depth slots, then one u64 per group:
 * the bytes it sent).  Returns SPLITZIP_OK or SPLITZIP_E_INVALID. */
int splitzip_pipeline_sizes(int dtype, size_t n_elems, uint32_t n_codebooks, size_t segment_elems,
                            size_t group_elems, uint32_t depth, size_t* d_work_bytes, size_t* h_link_bytes);

/* splitzip_pipeline_transfer: d_in (n_elems, device, 16-byte aligned) ->
 * d_out (device, 16-byte aligned).
 *   compress      1: groups travel compressed; 0: the raw groups travel the
 *                 same pipeline (the uncompressed baseline).
 *   d_work        device memory of d_work_bytes, 256-byte aligned.
 *   h_link        pinned host memory (hipHostMalloc with hipHostMallocCoherent,
 *                 so the encoder's size words reach the host at once) of
 *                 h_link_bytes, 256-byte aligned.
 *   d_status      optional device int32, as in splitzip_decompress.
 *   h_group_bytes optional host array of ceil(n / group_elems) entries: the
 *                 bytes each group sent over the link.
 *   streams       four distinct streams: encode, device-to-host copies,
 *                 host-to-device copies, decode.
 * Blocking: the calling thread drives the pipeline and returns after all four
 * streams are synchronized.  When no step can be queued it polls for 40 us,
 * then naps 20 us between polls; if no step can proceed for 60 s it returns
 * SPLITZIP_E_HIP.  The call creates 4 * depth HIP events (no timing) and
 * destroys them before it returns; it allocates no device or host buffer.
 * On an error return, work already queued may still run; synchronize the
 * streams before reusing the buffers.  Returns SPLITZIP_OK,
 * SPLITZIP_E_INVALID, SPLITZIP_E_CAPACITY, SPLITZIP_E_CODEBOOK or
 * SPLITZIP_E_HIP. */
int splitzip_pipeline_transfer(int dtype, const void* d_in, size_t n_elems, const uint8_t* h_codebooks,
                               uint32_t n_codebooks, size_t segment_elems, size_t group_elems, uint32_t depth,
                               int compress, void* d_work, size_t d_work_bytes, void* h_link, size_t h_link_bytes,
                               void* d_out, int32_t* d_status, uint64_t* h_group_bytes,
                               const hipStream_t streams[4]);

/* ---- 4-bit KV cache -------------------------------------------------------
 * Where the codec carries a cache to the decode side bit for bit, these calls
 * keep it there in 4 bits, attend over it and keep it within a budget.  The
 * cache is paged: splitzip_kv4_append puts K and V rows away (the encoder),
 * splitzip_kv4_read gives them back (the decoder), splitzip_kv4_attention
 * reads them in place and splitzip_kv4_evict drops the slots that drew the
 * least attention.
 *
 * Values.  The OCP microscaling form: E2M1 elements (0, 0.5, 1, 1.5, 2, 3, 4,
 * 6 and their negatives; code bit 3 is the sign) in blocks of 32 consecutive
 * channels of one token of one head, with one E8M0 scale byte s per block: a
 * value is element * 2^(s - 127).  The encoder takes the least exponent e with
 * max|x| < 7 * 2^e, s = e + 127 clamped to 1..252, and rounds every x / 2^e to
 * the nearest element, ties to the even code, beyond 6 to 6: no element is
 * further off than half its step (2^e at most), and no value of 252 or below
 * overflows BF16.
 *
 * A page holds page_tokens consecutive slots of every head; the bytes of one
 * head in it are contiguous (P = page_tokens, D = head_dim, 17/16 P D bytes,
 * even channel in a byte's low nibble):
 *   K codes   [P][D/2]
 *   V codes   [P/4][16][4][D/32]: token / 4, channel / (D/16), token % 4,
 *             bytes of the D/16 channels
 *   K scales  [P][D/32]
 *   V scales  [P/4][D/32][4]
 * d_pages is [n_pages][n_heads][splitzip_kv4_page_bytes].  Side arrays, where
 * a call takes them, are [n_pages][n_heads][page_tokens]: d_mass (float), the
 * attention weight a slot has drawn so far, and d_pos (int32), the position of
 * its token in the text (what the keys were rotated by, say).
 *
 * A batch names its sequences' pages by a block table and holds, packed one
 * sequence after the other, the rows that a call is about: sequence b has the
 * rows d_cu[b] .. d_cu[b + 1] - 1, which stand for its LAST slots, d_lens[b] -
 * (number of rows) up to d_lens[b] - 1.  d_lens counts the rows of the call.
 * Two sequences may share pages that are only read.  A sequence whose length,
 * rows or page numbers are out of range is reported through d_status
 * (SPLITZIP_E_CORRUPT, sticky as in splitzip_decompress) and its results are
 * unspecified or left as they were; every access stays inside the arrays.
 * Packed rows of no sequence are left as they were. */
typedef struct {
  void* d_pages;        /* 16-byte aligned */
  uint32_t n_pages;     /* 1 .. 2^31 - 1 */
  uint32_t n_heads;     /* KV heads, 1 .. 1024 */
  uint32_t head_dim;    /* 64, 128 or 256 */
  uint32_t page_tokens; /* 16, 32, 64, 128 or 256 */
} splitzip_kv4_cache;

typedef struct {
  const int32_t* d_table; /* [n_seqs][table_stride] page numbers */
  size_t table_stride;    /* entries between rows, >= ceil(max_len / page_tokens) */
  const int32_t* d_lens;  /* [n_seqs] slots in use */
  const int32_t* d_cu;    /* [n_seqs + 1] first packed row of each sequence; NULL: one row each (n_rows == n_seqs) */
  uint32_t n_seqs;        /* 0 .. 65535 */
  uint32_t max_len;       /* no length is larger; up to 2^23 */
  uint32_t max_new;       /* no sequence has more rows; 1 .. n_rows where there are rows */
  uint32_t n_rows;        /* rows of the packed tensors; up to 2^30 */
} splitzip_kv4_batch;

/* Element types of the 4-bit cache's rows besides splitzip_dtype. */
enum { SPLITZIP_KV4_FP16 = 3 };

/* Bytes of one head in one page, 0 for a head_dim or page_tokens outside the
 * lists above. */
size_t splitzip_kv4_page_bytes(uint32_t head_dim, uint32_t page_tokens);

/* Encode rows into the batch's slots.  One launch.
 *   dtype        SPLITZIP_BF16, SPLITZIP_KV4_FP16 or SPLITZIP_FP8_E5M2.
 *   d_k, d_v     [n_rows][n_heads][head_dim] with strides in elements between
 *                rows and between heads, multiples of 8 (channels contiguous);
 *                aligned to 8 elements.
 *   d_positions  optional [n_rows]: the tokens' positions for d_pos; NULL: the
 *                slot's number.
 *   d_mass       optional: the rows' slots are set to 0.
 *   d_pos        optional: the rows' slots get their positions.
 * A NaN is stored as 0 and an infinity as the block's largest magnitude (its
 * scale is that of the finite values); d_status then gets
 * SPLITZIP_E_NONFINITE unless it already holds an error.  A sequence with
 * more rows than slots is an error of the batch.  Two rows that meet in one
 * slot (pages shared by mistake) leave either's bytes.
 * Returns SPLITZIP_OK, SPLITZIP_E_INVALID or SPLITZIP_E_HIP. */
int splitzip_kv4_append(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch, int dtype, const void* d_k,
                        size_t k_row_stride, size_t k_head_stride, const void* d_v, size_t v_row_stride,
                        size_t v_head_stride, const int32_t* d_positions, float* d_mass, int32_t* d_pos,
                        int32_t* d_status, hipStream_t stream);

/* Decode the batch's slots into rows d_k, d_v [n_rows][n_heads][head_dim]
 * (contiguous, 16-byte aligned; either may be NULL).  dtype: SPLITZIP_BF16
 * (exact) or SPLITZIP_KV4_FP16 (exact from 2^-24 to 65504, rounded to nearest
 * or infinite outside).  A sequence with more rows than slots is an error of
 * the batch.  One launch.  Returns SPLITZIP_OK, SPLITZIP_E_INVALID or
 * SPLITZIP_E_HIP. */
int splitzip_kv4_read(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch, int dtype, void* d_k,
                      void* d_v, int32_t* d_status, hipStream_t stream);

/* Bytes of d_work of splitzip_kv4_attention (the partial results of the
 * splits of the long axis); with_mass: d_mass_out is given.  0 for arguments
 * that the call refuses. */
size_t splitzip_kv4_attention_work_bytes(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch,
                                         uint32_t n_q_heads, int with_mass);

/* Causal attention of packed queries over the cache, heads grouped: query
 * head a reads KV head a / (n_q_heads / n_heads).  Row i of the m rows of a
 * sequence of length n sees the slots j <= n - m + i; its own K and V are in
 * the cache (appended before).  With x_ij = scale * q_i . k_j,
 *   p_ij = exp(x_ij) / sum_j exp(x_ij),  out_i = sum_j p_ij v_j,
 *   lse_i = log sum_j exp(x_ij)
 * and a row that sees no slot (m > n) gives out 0 and lse -infinity.  m is 1
 * when tokens are generated one by one, a few when drafts are checked, long
 * for prompts and chunks of them.
 *   dtype      of d_q and d_out: SPLITZIP_BF16 or SPLITZIP_KV4_FP16.
 *   d_q        [n_rows][n_q_heads][head_dim] with strides in elements between
 *              rows and heads, multiples of 8; 16-byte aligned; not overlapped
 *              by what the call writes.
 *   n_q_heads  a multiple of n_heads, at most 64 query heads per KV head.
 *   scale      finite and above 0.
 *   d_out      [n_rows][n_q_heads][head_dim], contiguous, 16-byte aligned.
 *   d_lse      optional float [n_rows][n_q_heads].
 *   d_mass, d_mass_out  optional, both or none: for every slot of a sequence
 *              d_mass_out = d_mass + the sum of p over the sequence's rows and
 *              the head's queries; they may be one array.  Sums run in a fixed
 *              order: results repeat bit for bit.  Sequences that share pages
 *              here leave one of their sums in them.
 *   d_work     splitzip_kv4_attention_work_bytes bytes, 256-byte aligned,
 *              overwritten; calls that may overlap need one each.
 * Logits have to be finite in 32 bits.  Weights and sums are held in 32 bits;
 * for the product with V a weight counts with 16 bits, or, in BF16 calls with more than 64 rows (tokens x query heads
 * of a KV head; 16 where head_dim is 256), as BF16.  Only launches kernels, as the codec's
 * calls.  Returns SPLITZIP_OK, SPLITZIP_E_INVALID, SPLITZIP_E_CAPACITY (d_work
 * too small) or SPLITZIP_E_HIP. */
int splitzip_kv4_attention(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch, int dtype,
                           const void* d_q, size_t q_row_stride, size_t q_head_stride, uint32_t n_q_heads, float scale,
                           void* d_out, float* d_lse, const float* d_mass, float* d_mass_out, void* d_work,
                           size_t work_bytes, int32_t* d_status, hipStream_t stream);

/* Bytes of d_work of splitzip_kv4_evict, 0 for arguments that it refuses. */
size_t splitzip_kv4_evict_work_bytes(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch, uint32_t budget);

/* Cut every sequence longer than `budget` to `budget` slots, each head for
 * itself.  Kept are first the slots whose token position is below `sinks` or
 * at least d_next_pos[b] - recent (all ranking equal), then those of the largest
 * d_mass (a NaN ranks below -infinity), equal ones by the lowest slot.  Slots below the new
 * length stay where they are: in ascending order, the i-th dropped slot below
 * it receives the i-th kept slot at or beyond it (cache bytes, mass and
 * position).  Attention does not depend on the order of past slots, so only
 * those few tokens move; d_pos says which token a slot holds.
 *   batch       d_cu, max_new and n_rows are not read.
 *   sinks + recent <= budget, budget >= 1.
 *   d_mass, d_pos, d_mass_out, d_pos_out  16-byte aligned.
 *   d_next_pos  [n_seqs] position that the sequence's next token will have.
 *   d_lens_out  [n_seqs] min(length, budget); may be d_lens.
 *   d_mass_out, d_pos_out  the slots below the new length; may be d_mass,
 *               d_pos.  Other entries are left as they were.
 *   d_work      splitzip_kv4_evict_work_bytes bytes, 256-byte aligned,
 *               overwritten; calls that may overlap need one each.
 * The sequences' pages must not be shared.  Returns SPLITZIP_OK,
 * SPLITZIP_E_INVALID, SPLITZIP_E_CAPACITY or SPLITZIP_E_HIP. */
int splitzip_kv4_evict(const splitzip_kv4_cache* cache, const splitzip_kv4_batch* batch, uint32_t budget,
                       uint32_t sinks, uint32_t recent, const int32_t* d_next_pos, const float* d_mass,
                       const int32_t* d_pos, int32_t* d_lens_out, float* d_mass_out, int32_t* d_pos_out, void* d_work,
                       size_t work_bytes, int32_t* d_status, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SPLITZIP_H */
