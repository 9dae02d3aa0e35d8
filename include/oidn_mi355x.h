/*
 * oidn_mi355x.h -- C ABI of the MI355X (gfx950) OIDN-style UNet denoiser.
 *
 * Pages cited (by title and symbol):
 *   [web-0.4]    "oidn-web 0.3.4 -> 0.4.0", nativeUNet.ts
 *   [web-0.5]    "oidn-web 0.4.0 -> 0.5.0", nativeUNet.ts
 *   [webgpu-0.6] "oidn-webgpu 0.0.0-stage -> 0.6.0", native/denoise.ts
 *
 * Conventions shared by every call
 *   - Images and activations are NHWC with batch 1.  Activations keep their
 *     channels in 4-lane blocks ([web-0.4] blocksForChannels,
 *     activationByteSize): a tensor of C logical channels stores
 *     C_store = 4 * ceil(C / 4) values per pixel and the unused lanes are 0.
 *   - Tensor pointers are DEVICE pointers owned by the caller.  Host pointers
 *     are named *_host.  The library never allocates or frees device memory
 *     and never synchronises, except the two weight-pack calls, which copy
 *     from host memory and wait for that copy.
 *   - Device work is enqueued on the given stream (0 = the null stream) and
 *     the call returns at once.
 *   - Every call returns an int status: OIDN_OK (0) or a negative code.  On
 *     any error nothing is enqueued and outputs are untouched;
 *     oidn_last_error() returns the message (thread-local).
 *   - dtype selects the storage type of activations and weights: OIDN_F16
 *     (fp16 storage, fp32 accumulate, MFMA path), OIDN_BF16 (bf16 storage,
 *     the same kernels with the bf16 MFMA; every stored value rounded to
 *     nearest even from fp32, as fp16 is) or OIDN_F32 (fp32 storage and
 *     arithmetic).  A conv's 16-bit output has its input's type; any 16-bit
 *     path may write fp32 instead.  Weights are packed for one dtype.
 *     Biases are always fp32 ([web-0.4] packConvTensors keeps the bias in f32).
 *   - Overlapping calls on different streams that share buffers race; the
 *     caller orders them.
 */
#ifndef OIDN_MI355X_H
#define OIDN_MI355X_H

#include <stddef.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define OIDN_OK              0
#define OIDN_E_INVALID      -1  /* null pointer, bad size, bad enum          */
#define OIDN_E_UNSUPPORTED  -2  /* valid request the library does not handle */
#define OIDN_E_WORKSPACE    -3  /* workspace or output capacity too small    */
#define OIDN_E_HIP          -4  /* a HIP runtime call or launch failed       */

/* ---- storage types ----------------------------------------------------- */
#define OIDN_F32   0
#define OIDN_F16   1
#define OIDN_BF16  2

/* ---- conv flags -------------------------------------------------------- */
#define OIDN_RELU     1u  /* y = max(y, 0) ([web-0.4] activationExpression)            */
#define OIDN_POOL2X2  2u  /* 2x2/2 max-pool fused after bias+ReLU; output h/2 x w/2
                             ([web-0.4] createFusedConvPoolShader)                    */

/* ---- HDR transfer ------------------------------------------------------ */
#define OIDN_TRANSFER_PU   0  /* named by [webgpu-0.6]; formula not on the pages:
                                 OIDN_E_UNSUPPORTED                                   */
#define OIDN_TRANSFER_LOG  1  /* F(x) = ln(1 + x), F^-1(y) = exp(y) - 1 (reading)    */

/* ---- norms around a block ------------------------------------------------ */
#define OIDN_NORM_NONE   0  /* the row itself                                  */
#define OIDN_NORM_RMS    1  /* x / sqrt(mean(x^2) + eps)                       */
#define OIDN_NORM_LAYER  2  /* (x - mean) / sqrt(mean((x - mean)^2) + eps)     */

/* ---- activations of the dense operators ---------------------------------- */
#define OIDN_ACT_NONE  0
#define OIDN_ACT_RELU  1   /* max(z, 0), slope 0 at 0                          */
#define OIDN_ACT_SILU  2   /* z / (1 + exp(-z))                                */
#define OIDN_ACT_GELU  3   /* z (1 + erf(z / sqrt 2)) / 2                      */

/* ---- flags of the dense operators ---------------------------------------- */
#define OIDN_X_CKPT8  1u   /* x is a checkpoint (oidn_ckpt_pack), its pitch unused */
#define OIDN_Z_CKPT8  2u   /* z is held in 8 bits                              */
#define OIDN_FP8_SQUARE  4u  /* a scale for 128 x 128 values (weights)          */
#define OIDN_X_FP8    8u   /* x is packed (oidn_fp8_pack), its pitch unused    */

/* ---- limits ------------------------------------------------------------ */
#define OIDN_MAX_SOURCE_CHANNELS 256   /* logical channels per conv source */
#define OIDN_MAX_OUT_CHANNELS    128
#define OIDN_TILE_ALIGN           16   /* tile starts and sizes (four 2x2 pools) */
#define OIDN_DEFAULT_OVERLAP      96   /* alignUp(one-sided receptive reach 94, 16) */

/* One tile of a tile grid: the input rectangle the network runs on and the
 * output rectangle it writes ([webgpu-0.6] recordDenoiseExecution reads
 * tile.input.{x,y,width,height} and tile.output.{x,y,width,height}).
 * Input rectangles may extend past the image: those reads clamp to the edge. */
typedef struct oidn_tile {
  int in_x, in_y, in_w, in_h;
  int out_x, out_y, out_w, out_h;
} oidn_tile;

/* Message of the last failed call on this thread ("" if none). */
const char* oidn_last_error(void);

/* ABI version: major * 10000 + minor * 100 + patch. */
int oidn_version(void);

/* ========================================================================
 * 3x3 convolution, stride 1, zero padding 1, bias, optional ReLU and fused
 * 2x2 max-pool ([web-0.4] createConvShader: the sum starts at the bias and
 * skips taps outside the image; createFusedConvPoolShader).
 *
 *   y[p][o] = act(b[o] + sum_{ky,kx in 0..2} sum_i W[o][ky][kx][i] * x[p + (ky-1, kx-1)][i])
 *
 * Weights are OHWI float32 over LOGICAL input channels.  A conv over two
 * sources (the decoder's upsample + concat) indexes the logical concat
 * [upsampled source (cin0 channels), skip (cin1 channels)].
 * ======================================================================== */

/* Bytes of the packed weights+bias buffer for (cin0, cin1, cout, dtype).
 * cin1 = 0 for a one-source conv.  Host only. */
int oidn_conv3x3_weights_bytes(int cin0, int cin1, int cout, int dtype, size_t* bytes);

/* Packs OHWI float32 weights (cout x 3 x 3 x (cin0 + cin1), host) and a
 * float32 bias (cout, host) into the device layout of the chosen dtype
 * (fp16 and bf16: MFMA A-operand fragments in K-major chunk order, pad lanes 0, the
 * upsampled source of a two-source conv as four sums of ky rows -- W0,
 * W1 + W2, W0 + W1, W2, each rounded once to the storage type -- because an output row
 * reads only two low-resolution rows of it; fp32: [out block][tap][stored
 * input channel][4 out lanes]).  d_packed must hold
 * oidn_conv3x3_weights_bytes() bytes.  Blocks until the upload finished.
 * Two sources need cin0 % 4 == 0 (each source keeps its own 4-lane blocks,
 * [web-0.4] createTiledDecoderShader). */
int oidn_conv3x3_pack_weights(const float* w_ohwi_host, const float* bias_host,
                              int cin0, int cin1, int cout, int dtype,
                              void* d_packed, hipStream_t stream);

/* Same packing into host memory (host_packed: oidn_conv3x3_weights_bytes()
 * bytes), no device work.  For inspecting or caching the packed layout. */
int oidn_conv3x3_pack_weights_host(const float* w_ohwi_host, const float* bias_host,
                                   int cin0, int cin1, int cout, int dtype, void* host_packed);

/* One-source conv.  x: h x w x C_store(cin) of in_dtype; y: (h x w, or
 * h/2 x w/2 with OIDN_POOL2X2) x C_store(cout) of out_dtype.  in_dtype f32
 * needs out_dtype f32; in_dtype f16 allows f16 or f32 out.  POOL2X2 needs even
 * h and w.  w_packed from oidn_conv3x3_pack_weights(cin, 0, cout, in_dtype).
 * x and y must not overlap. */
int oidn_conv3x3(const void* x, int h, int w, int cin, const void* w_packed,
                 void* y, int cout, int in_dtype, int out_dtype, unsigned flags,
                 hipStream_t stream);

/* Decoder conv: nearest 2x upsample of `low` (h/2 x w/2 x c_low) concatenated
 * with `skip` (h x w x C_store(c_skip)), never materialised ([web-0.4]
 * createTiledDecoderShader reads the upsampled source at (x/2, y/2); blocks
 * of the first source come first).  h, w even; c_low % 4 == 0.  w_packed from
 * oidn_conv3x3_pack_weights(c_low, c_skip, cout, in_dtype). */
int oidn_conv3x3_upcat(const void* low, int c_low, const void* skip, int c_skip,
                       int h, int w, const void* w_packed, void* y, int cout,
                       int in_dtype, int out_dtype, unsigned flags, hipStream_t stream);

/* Two convs in one pass, y = convB(relu(convA(x))), the 32-channel
 * intermediate never leaving the chip: convA is cin -> 32 (bias, ReLU,
 * fp16 rounding as oidn_conv3x3 with OIDN_RELU), convB is 32 -> cout with
 * `flags` and `out_dtype` as in oidn_conv3x3.  Both convs as defined by
 * [web-0.4] createConvShader ("oidn-web 0.3.4 -> 0.4.0", nativeUNet.ts);
 * the fusion is this library's.  fp16 storage only.  wa_packed / wb_packed:
 * oidn_conv3x3_pack_weights output for (cin, 0, 32) and (32, 0, cout).
 * x: h x w x 4 ceil(cin / 4) fp16; y as oidn_conv3x3's output.  The result
 * equals oidn_conv3x3(convB) applied to oidn_conv3x3(convA) bit for bit.
 * Needs 4 ceil(cin / 4) a multiple of 8 and either <= 32 or a multiple of
 * 32, and cout <= 32 (else OIDN_E_UNSUPPORTED). */
int oidn_conv3x3_pair(const void* x, int h, int w, int cin, const void* wa_packed,
                      const void* wb_packed, void* y, int cout, int out_dtype, unsigned flags,
                      hipStream_t stream);

/* Name of the kernel instance that oidn_conv3x3 (cin1 == 0) or
 * oidn_conv3x3_upcat (cin0 = c_low, cin1 = c_skip) runs for this shape,
 * written NUL-terminated into buf (cap bytes), e.g.
 * "conv3x3_f16_mfma<4, 8, 4, false>"; *blocks (may be null) receives the
 * launch's workgroup count.  Same validation as those calls; host only. */
int oidn_conv3x3_kernel(int h, int w, int cin0, int cin1, int cout, int in_dtype,
                        int out_dtype, unsigned flags, char* buf, int cap, int* blocks);

/* ========================================================================
 * Elementwise and gather passes
 * ======================================================================== */

/* 2x2 max-pool, stride 2 ([web-0.4] createMaxPoolShader; [web-0.5] coalesced
 * "channels" layout).  x: h x w x C_store(c); y: h/2 x w/2 x C_store(c).
 * h and w must be even. */
int oidn_pool2x2(const void* x, int h, int w, int c, void* y, int dtype, hipStream_t stream);

/* Materialised nearest 2x upsample + concat: z[y][x] = [low[y/2][x/2] (C_store(c_low)
 * lanes), skip[y][x] (C_store(c_skip) lanes)].  low: h/2 x w/2; skip, z: h x w.
 * h, w even; c_low % 4 == 0. */
int oidn_upsample_concat(const void* low, int c_low, const void* skip, int c_skip,
                         int h, int w, void* z, int dtype, hipStream_t stream);

/* Input pass of one tile ([webgpu-0.6] inputShader; lane layout of [web-0.4]
 * createInputPackShader).  color/albedo/normal: img_h x img_w RGBA float32
 * (16 B per pixel); albedo and normal may be NULL (3 or 6 channels; normal
 * needs albedo).  For each tile pixel (tx, ty) the source pixel is
 * clamp((tile_x + tx, tile_y + ty), (0, 0), (img_w-1, img_h-1)).  Colour:
 * hdr ? F(sanitize(rgb * input_scale, 0, FLT_MAX)) : sanitize(rgb, 0, 1);
 * albedo: sanitize(rgb, 0, 1); normal: sanitize(rgb, -1, 1) * 0.5 + 0.5,
 * where sanitize maps NaN to 0 and clamps.  The 3/6/9 channels are packed
 * densely into 4-lane blocks (lane l of block b is channel 4b + l), unused
 * lanes 0.  packed: tile_h x tile_w x C_store(channels) of dtype.
 * tile_w * tile_h above 2^31 - 1025 pixels: OIDN_E_UNSUPPORTED. */
int oidn_pack_input(const float* color, const float* albedo, const float* normal,
                    int img_w, int img_h, int tile_x, int tile_y, int tile_w, int tile_h,
                    int hdr, int transfer, float input_scale, void* packed, int dtype,
                    hipStream_t stream);

/* Output pass of one tile ([webgpu-0.6] outputShader).  net_rgba: the
 * network's RGBA float32 output for a tile_w x tile_h tile.  For each pixel
 * (x, y) of the out_w x out_h output rectangle:
 *   d = sanitize(net[y + in_off_y][x + in_off_x].rgb, 0, hdr ? FLT_MAX : 1)
 *   out[out_y + y][out_x + x] = (hdr ? F^-1(d) / input_scale : d,
 *                                color[out_y + y][out_x + x].a)
 * out_rgba: img_h x img_w RGBA float32; only the rectangle is written.
 * out_w * out_h above 2^31 - 1025 pixels: OIDN_E_UNSUPPORTED. */
int oidn_unpack_output(const float* net_rgba, int tile_w, int tile_h, int in_off_x,
                       int in_off_y, const float* color, int img_w, int img_h, int out_x,
                       int out_y, int out_w, int out_h, int hdr, int transfer,
                       float input_scale, float* out_rgba, hipStream_t stream);

/* ========================================================================
 * Tile grid (host only, pure).  [webgpu-0.6] recordDenoiseExecution plans
 * tiles with maxTileSize (0 = the whole image, aligned up) and an overlap
 * from the receptive field aligned to the tile alignment; the planner body
 * is not on the pages.  Reading: per axis of extent E with tile limit T and
 * overlap O, one tile when alignUp(E, 16) <= T, else n = ceil(E / (T - 2O))
 * output spans of S = alignUp(ceil(E / n), 16) pixels whose input spans are
 * min(S + 2O, alignUp(E, 16)) wide, shifted to stay in [0, alignUp(E, 16)).
 * Tiles are listed row-major (y outer).  max_tile must be 0 or a multiple of
 * 16; overlap < 0 selects OIDN_DEFAULT_OVERLAP, otherwise a multiple of 16.
 * *count receives the number of tiles; OIDN_E_WORKSPACE if it exceeds cap
 * (tiles may be NULL with cap 0 to query the count).
 * ======================================================================== */
int oidn_plan_tiles(int w, int h, int max_tile, int overlap, oidn_tile* tiles, int cap,
                    int* count);

/* ========================================================================
 * UNet.  Sixteen 3x3 convs in this order (logical channels; the pages'
 * modelSpec is not shown -- wiring read from the OIDN-style channel list):
 *   enc_conv0 in->32, enc_conv1 32->32 +pool, enc_conv2 32->48 +pool,
 *   enc_conv3 48->64 +pool, enc_conv4 64->80 +pool, enc_conv5a 80->96,
 *   enc_conv5b 96->96, dec_conv4a [up(5b) 96 | pool3 64]->112, dec_conv4b
 *   112->112, dec_conv3a [up 112 | pool2 48]->96, dec_conv3b 96->96,
 *   dec_conv2a [up 96 | pool1 32]->64, dec_conv2b 64->64, dec_conv1a
 *   [up 64 | input in]->64, dec_conv1b 64->32, dec_conv0 32->3 (no ReLU,
 *   float32 RGBA output, lane 3 = 0).
 * in_channels is 3, 6 or 9 ([web-0.4] NativeUNetExecutor constructor).
 * ======================================================================== */

int oidn_unet_layer_count(void);

/* Shape of layer `layer` (0..15): logical channels of the (upsampled) source
 * and of the skip (0 if none), output channels, resolution level (0 = full,
 * 1 = /2, ...), flags (OIDN_RELU | OIDN_POOL2X2), and a static name. */
int oidn_unet_layer_info(int in_channels, int layer, int* cin0, int* cin1, int* cout,
                         int* level, unsigned* flags, const char** name);

/* Name of the kernel instance that runs `layer` on `batch` tw x th tiles per
 * launch (oidn_unet_tile_batch; the launch plan counts the whole launch's
 * workgroups) (for matching per-kernel timings and profiles), written NUL-terminated into
 * buf (cap bytes), e.g. "conv3x3_f16_mfma<2, 16, 2, false>" (fragments and
 * rows per wave, row groups, fp32 output) or, for both layers of a fused
 * pair, "conv3x3_pair_f16<2, 2, 0, 3>" (convA channel groups, convB
 * fragments, output: 0 16-bit, 1 fp32, 2 straight through the output pass;
 * input: bit 0 tap-packed, bit 1 the caller's images through the input pass),
 * or "conv3x3_ws_f16<4, 8, 4, false>" for a layer whose whole weight set fits
 * in LDS (dec_conv1a with the tap-packed skip): one persistent workgroup per
 * compute unit that walks the launch's tiles, so *blocks is that grid;
 * with bf16 storage "conv3x3_bf16_mfma", "conv3x3_pair_bf16" and
 * "conv3x3_ws_bf16".  *blocks receives the launch's workgroup count.  Host
 * only. */
int oidn_unet_layer_kernel(int in_channels, int layer, int tw, int th, int batch, int dtype,
                           char* buf, int cap, int* blocks);

/* Bytes of the packed weights of all sixteen layers.  With 9 input channels
 * on the 16-bit paths the blob also holds a second copy of enc_conv0's and
 * dec_conv1a's weights in the layout oidn_unet_forward uses for its
 * tap-packed input (channel 8's row neighbours beside it: half the matrix
 * steps for that source); oidn_unet_forward_packed uses the plain copies.
 * On the 16-bit paths dec_conv0's one output fragment holds its three output
 * channels' weights and biases in each of its four 4-channel groups (lanes
 * 4g .. 4g + 2, lane 4g + 3 zero), so the output pass fused into that
 * layer's kernel can spread its rows over all lanes; the size is unchanged. */
int oidn_unet_weights_bytes(int in_channels, int dtype, size_t* bytes);

/* Packs all layers: w_ohwi_host[i] is cout x 3 x 3 x cin (cin = cin0 + cin1
 * of layer i), bias_host[i] is cout floats.  Blocks until uploaded. */
int oidn_unet_pack_weights(const float* const* w_ohwi_host, const float* const* bias_host,
                           int in_channels, int dtype, void* d_weights, hipStream_t stream);

/* Workspace for oidn_unet_forward_packed on a tw x th tile (liveness-planned
 * activation buffers; input and output are the caller's). */
int oidn_unet_packed_workspace_bytes(int in_channels, int tw, int th, int dtype, size_t* bytes);

/* The network on one packed tile ([web-0.4] NativeUNetExecutor.execute: one
 * pass per node, the last writing float32).  packed_in: th x tw x
 * C_store(in_channels) of dtype (from oidn_pack_input); net_out_rgba: th x tw
 * x 4 float32.  tw, th: positive multiples of 16. */
int oidn_unet_forward_packed(const void* d_weights, int in_channels, const void* packed_in,
                             int tw, int th, void* workspace, size_t ws_bytes,
                             float* net_out_rgba, int dtype, hipStream_t stream);

/* Workspace for oidn_unet_forward on a w x h image with this tile plan
 * (on the 16-bit paths one copy of the per-tile plan for each tile of a batch,
 * see oidn_unet_tile_batch). */
int oidn_unet_workspace_bytes(int in_channels, int w, int h, int max_tile, int overlap,
                              int dtype, size_t* bytes);

/* Tiles of this plan that oidn_unet_forward runs through the network
 * together: on the 16-bit paths, where both image passes run inside the first
 * and last convs, up to 16 consecutive tiles of one size share one launch
 * per layer (tile index in grid z, or one tile sequence for the persistent
 * weight-stationary layer); else 1.  The per-kernel events of
 * oidn_unet_forward_timed cover the first such batch.  Host only. */
int oidn_unet_tile_batch(int in_channels, int w, int h, int max_tile, int overlap, int dtype,
                         int* batch);

/* Where oidn_unet_forward keeps the packed network input of a tile inside
 * its workspace (host only; for inspection and tests): tile k of the last
 * tile batch of the call (oidn_unet_tile_batch) at workspace + *offset +
 * k * *tile_stride (stride 0 when tiles run one by one), tile_h x tile_w
 * pixels of *lanes values of dtype.  With *taps (16-bit storage, nine
 * channels) lanes 0..7 hold channels 0..7, lanes 8, 9, 10 channel 8 of the
 * pixels in tile columns x - 1, x, x + 1 (zero past the tile's edge), the
 * rest zero; else the oidn_pack_input layout padded with zero lanes.  The
 * values stay there after the call until the workspace is reused. */
int oidn_unet_input_layout(int in_channels, int w, int h, int max_tile, int overlap, int dtype,
                           size_t* offset, size_t* tile_stride, int* lanes, int* taps);

/* End-to-end denoise ([webgpu-0.6] recordDenoiseExecution): plan the tile
 * grid, then for each tile in order: input pass, network, output pass into
 * the tile's output rectangle of out_rgba (h x w RGBA float32; on the 16-bit
 * path the network's first fused pair runs the input pass on the images and
 * the last writes that rectangle itself).  in_channels
 * must match the non-NULL images (color; + albedo; + normal). */
int oidn_unet_forward(const void* d_weights, int in_channels, const float* color,
                      const float* albedo, const float* normal, int w, int h, int hdr,
                      int transfer, float input_scale, int max_tile, int overlap,
                      void* workspace, size_t ws_bytes, float* out_rgba, int dtype,
                      hipStream_t stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): the same
 * denoise as oidn_unet_forward, with no workspace argument.  Its workspace is
 * a static device array of OIDN_NOALLOC_SCRATCH_MB MiB inside the library,
 * one per GPU, held until the process ends; the call allocates and frees
 * nothing.  As many tiles run per launch as that array holds (the results
 * are the same bits as oidn_unet_forward's).  A plan whose single tile needs
 * more (oidn_unet_workspace_bytes / oidn_unet_tile_batch) is refused with
 * OIDN_E_WORKSPACE before any device work: 1920x1080 in one tile needs about
 * 400 MB, so such images need max_tile (512 fits).  Nothing in the array
 * needs to start at zero (every value is written before it is read).  All
 * calls on one GPU share the array: calls that overlap in time on one GPU
 * (other streams, other host threads) race and must be ordered by the
 * caller. */
#define OIDN_NOALLOC_SCRATCH_MB 64
int oidn_unet_forward_noalloc(const void* d_weights, int in_channels, const float* color,
                              const float* albedo, const float* normal, int w, int h, int hdr,
                              int transfer, float input_scale, int max_tile, int overlap,
                              float* out_rgba, int dtype, hipStream_t stream);

/* Size in bytes of the array oidn_unet_forward_noalloc uses.  Host only. */
int oidn_unet_noalloc_scratch_bytes(size_t* bytes);

/* Same as oidn_unet_forward, and records events[k] on the stream before the
 * k-th kernel of the FIRST tile or tile batch (k = 0: input pass, 1..16: layers, 17: output
 * pass) and events[18] after it, for per-kernel timing.  Where the first
 * layer's kernel runs the input pass itself (layer kernel input bit 1),
 * events[0] and events[1] are recorded back to back; where the last layer's
 * runs the output pass (output field 2), events[17] and events[18].
 * n_events >= 19; events are hipEvent_t handles (see oidn_event_create). */
int oidn_unet_forward_timed(const void* d_weights, int in_channels, const float* color,
                            const float* albedo, const float* normal, int w, int h, int hdr,
                            int transfer, float input_scale, int max_tile, int overlap,
                            void* workspace, size_t ws_bytes, float* out_rgba, int dtype,
                            hipStream_t stream, void* const* events, int n_events);

/* ========================================================================
 * Dense operators over activation rows.  An NHWC activation of h x w pixels
 * is a matrix of m = h * w rows of channels; its row pitch (`ld...`, in
 * elements, >= the row's columns) is the stored channel count, so any run of
 * channels of a wider tensor is a matrix too.  Weights are row-major with one
 * row per output channel, in dtype; biases and their gradients are float32.
 * Sums, activations and slopes are fp32; every output is rounded once, to
 * nearest even, where it is stored.  fp16 outputs beyond 65504 become
 * infinite, and so do what passes from one product to the next in fp16 (h, dz,
 * da, db); with OIDN_F32 nothing is rounded on the way.  Results do not depend on timing: a call with the same arguments
 * gives the same bits.
 *
 * Any size and pitch works and any element-aligned base; bases and pitches
 * that are multiples of 16 bytes are fastest.  m may be 0 (sums over no rows
 * are 0, nothing else is written).  Outputs must not overlap inputs, except
 * that `residual` may be y and `add` may be dx (same pitch).  Columns between
 * a row's end and its pitch are never written; they may be read, and what they
 * hold does not matter.  Column counts
 * above 2^24, matrices above 2^38 elements and products of more tiles than a
 * launch holds (about 2^24; of 64 x 64 where a side is short):
 * OIDN_E_UNSUPPORTED.
 *
 * The workspace (16-byte aligned, the size the matching *_workspace_bytes
 * call gives) holds nothing between calls.
 * ======================================================================== */

/* 8-bit activation checkpoints: what a forward pass keeps for its backward
 * pass, at half the bytes of a 16-bit type.  A row's columns go in blocks of
 * 32 that share a scale:
 *   s = bf16(max|x| / 127),  q = rint(x / s) in [-127, 127],  value = q s.
 * Layout of an m x n checkpoint: m rows of int8 codes, padded to whole blocks
 * (padding holds 0), then one bf16 scale per row and block.  Blocks with
 * s < 2^-120 are stored as zeros; a block with an infinity or a NaN reads back
 * as NaN.  A finite value of a 16-bit type reads back finite in it: one that the
 * rounding of s carries past the range becomes the largest.  The buffer is 16-byte aligned. */
int oidn_ckpt_bytes(long m, long n, size_t* bytes);
int oidn_ckpt_pack(const void* x, long ldx, long m, long n, void* ckpt, int dtype,
                   hipStream_t stream);
int oidn_ckpt_unpack(const void* ckpt, long m, long n, void* y, long ldy, int dtype,
                     hipStream_t stream);

/* Dense layer (a 1 x 1 convolution):
 *   z = x w^T + bias,  y = act(z) + residual
 * x: m x k, w: n x k, bias: n floats or NULL, residual: m x n or NULL, y: m x n.
 * z, if not NULL, receives the pre-activation for the backward pass: m x n of
 * dtype at pitch ldz or, with OIDN_Z_CKPT8, a checkpoint of it. */
int oidn_linear_workspace_bytes(long m, int k, int n, int dtype, size_t* bytes);
int oidn_linear(const void* x, long ldx, const void* w, long ldw, const float* bias,
                const void* residual, long ldr, void* y, long ldy, void* z, long ldz, long m, int k,
                int n, int act, int dtype, unsigned flags, void* workspace, size_t ws_bytes,
                hipStream_t stream);

/* Its gradients, from dy (m x n):
 *   dz = dy act'(z),  dx = dz w,  dw = dz^T x,  dbias = sum of dz's rows
 * (the residual's gradient is dy itself; dz, and an x read from 8 bits, are
 * rounded to dtype before the products).  dx, dw and dbias may each be NULL.
 * z as saved by oidn_linear (unused with OIDN_ACT_NONE); x as given to it, or
 * with OIDN_X_CKPT8 a checkpoint of it. */
int oidn_linear_backward_workspace_bytes(long m, int k, int n, int act, int dtype, unsigned flags,
                                         size_t* bytes);
int oidn_linear_backward(const void* dy, long lddy, const void* x, long ldx, const void* z, long ldz,
                         const void* w, long ldw, void* dx, long lddx, void* dw, long lddw,
                         float* dbias, long m, int k, int n, int act, int dtype, unsigned flags,
                         void* workspace, size_t ws_bytes, hipStream_t stream);

/* Gated feed-forward block over rows of d channels with f hidden ones:
 *   [a | b] = x w_in^T + b_in,  h = act(a) * b,  y = h w_out^T + b_out + residual
 * w_in: 2f x d (the f gate rows, then the f up rows), w_out: d x f, both
 * contiguous; b_in (2f), b_out (d) and residual (m x d) may be NULL.  h is
 * rounded to dtype between the two products.  z, if not NULL, receives [a | b]
 * for the backward pass: m x 2f of dtype, contiguous, or with OIDN_Z_CKPT8 two
 * m x f checkpoints one after the other (a, then b; 2 oidn_ckpt_bytes(m, f)). */
int oidn_ffn_workspace_bytes(long m, int d, int f, int dtype, size_t* bytes);
int oidn_ffn(const void* x, long ldx, const void* w_in, const float* b_in, const void* w_out,
             const float* b_out, const void* residual, long ldr, void* y, long ldy, void* z, long m,
             int d, int f, int act, int dtype, unsigned flags, void* workspace, size_t ws_bytes,
             hipStream_t stream);

/* Its gradients, from dy (m x d):
 *   dh = dy w_out,  da = dh b act'(a),  db = dh act(a),
 *   dx = [da | db] w_in + add,  dw_in = [da | db]^T x,  dw_out = dy^T h,
 *   db_in = sum of [da | db]'s rows,  db_out = sum of dy's rows
 * add (m x d or NULL) is what else reaches x: dy where x is also the residual.
 * da, db, h and an x read from 8 bits are rounded to dtype before the products
 * that read them.  Any of dx, dw_in, db_in, dw_out, db_out may be NULL. */
int oidn_ffn_backward_workspace_bytes(long m, int d, int f, int dtype, unsigned flags, size_t* bytes);
int oidn_ffn_backward(const void* dy, long lddy, const void* x, long ldx, const void* z,
                      const void* w_in, const void* w_out, const void* add, long ldadd, void* dx,
                      long lddx, void* dw_in, float* db_in, void* dw_out, float* db_out, long m, int d,
                      int f, int act, int dtype, unsigned flags, void* workspace, size_t ws_bytes,
                      hipStream_t stream);

/* Dense layer in 8-bit floating point, with a scale for each block of 128 summed
 * values.  Packed form of an m x n matrix: e4m3 codes (4 exponent bits, 3 mantissa
 * bits, largest 448), then a scale 2^e per row and block of 128 columns,
 *   e the least whole number with max|x| <= 448 2^e, held in [-120, 120],
 *   code = x 2^-e rounded to nearest even, value = code 2^e.
 * The scale is a power of two: it costs no precision, and the matrix cores apply it.
 * Infinities and NaN become NaN, and the scale is that of the finite values.
 * Layout: m rows of codes, padded with zeros to whole blocks; then for each row a
 * byte e + 127 per block, padded to whole words of four bytes.  16-byte aligned.
 * oidn_fp8_pack makes the packed form of x (m x n) and / or of its transpose (n x m,
 * blocks of 128 rows of x): one of the two may be NULL.  With OIDN_FP8_SQUARE each
 * 128 x 128 values share a scale, so that both hold the same values: for weights,
 * which a forward pass sums over one way and a backward pass the other.
 * oidn_fp8_unpack gives the values; a finite one that the rounding carried past the
 * range of dtype becomes the largest. */
int oidn_fp8_bytes(long m, long n, size_t* bytes);
int oidn_fp8_pack(const void* x, long ldx, long m, long n, void* packed, void* packed_t, int dtype,
                  unsigned flags, hipStream_t stream);
int oidn_fp8_unpack(const void* packed, long m, long n, void* y, long ldy, int dtype, hipStream_t stream);

/* The layer of oidn_linear on packed values:
 *   z = [x] [w]^T + bias,  y = act(z) + residual,  [.] the packed form's values
 * w8: the packed weights (n x k).  x: m x k of dtype, packed inside, or with
 * OIDN_X_FP8 a packed matrix.  dtype: OIDN_F16 or OIDN_BF16.  The products of codes
 * are added eight neighbours at a time, and what lies below 2^-13 of the largest one's
 * power of two is cut off: each eight is off by less than 7 2^-13 of its largest product.
 * Those sums are added in fp32.  Of normal data 1e-5 to 4e-5 of a result, far below the
 * storage type's rounding; where large products cancel it may be all of what is left
 * (oidn_linear adds in fp32 throughout).
 * Faster than oidn_linear where a layer is large (8192 -> 8192 at any rows, 4096 -> 4096
 * from 512 rows on) or x is packed already; no faster up to 1024 -> 1024 with x not packed,
 * and slower with at most 128 inputs.
 * k, n <= 2^23.  The rest is as for oidn_linear. */
int oidn_linear_fp8_workspace_bytes(long m, int k, int n, int dtype, unsigned flags, size_t* bytes);
int oidn_linear_fp8(const void* x, long ldx, const void* w8, const float* bias, const void* residual,
                    long ldr, void* y, long ldy, void* z, long ldz, long m, int k, int n, int act,
                    int dtype, unsigned flags, void* workspace, size_t ws_bytes, hipStream_t stream);

/* Its gradients, with dz = dy act'(z) not rounded before it is coded:
 *   dx = [dz] [w],  dw = [dz^T] [x^T]^T,  dbias = sum of dz's rows
 * [dz]: blocks of 128 along a row; [dz^T], [x^T]: blocks of 128 rows of a column.
 * w8t: the packed transpose of w (k x n), of the same call with OIDN_FP8_SQUARE as the
 * forward pass's w8.  x: m x k of dtype, or with OIDN_X_FP8 its packed transpose
 * (k x m), which a forward pass may keep in place of x.  m <= 2^23. */
int oidn_linear_fp8_backward_workspace_bytes(long m, int k, int n, int act, int dtype, unsigned flags,
                                             size_t* bytes);
int oidn_linear_fp8_backward(const void* dy, long lddy, const void* x, long ldx, const void* z, long ldz,
                             const void* w8t, void* dx, long lddx, void* dw, long lddw, float* dbias,
                             long m, int k, int n, int act, int dtype, unsigned flags, void* workspace,
                             size_t ws_bytes, hipStream_t stream);

/* ========================================================================
 * What stands around a block over activation rows: the norm before it, and the
 * residual sum after it with a norm, a gate, a residual scale and dropout.
 * Matrices, pitches and types are as above; weights, shifts, gates and their
 * gradients are float32.  Statistics and sums are fp32; every output is rounded
 * once.  Rows of n columns, each by itself: a NaN or an infinity stays in its row.
 * A row whose sum of squares passes the range of float32 becomes zeros or NaN; so,
 * where eps is 0, does one whose sum falls below it, as of equal values (of zeros, with
 * OIDN_NORM_RMS).
 * In place: y of oidn_norm may be x, u may be x or o, y of oidn_dropout may be x
 * or the residual, add may be dx (same pitch).
 * ======================================================================== */

/* Before a block:  y = norm(x) weight + shift.  weight and shift (n floats) may
 * be NULL: 1 and 0.  norm: OIDN_NORM_RMS or OIDN_NORM_LAYER. */
int oidn_norm(const void* x, long ldx, const float* weight, const float* shift, void* y, long ldy, long m,
              int n, int norm, float eps, int dtype, hipStream_t stream);

/* Its gradients, from dy: with hat = norm(x) = (x - mean) r and g = dy weight,
 *   dx = r (g - mean(g) - hat mean(g hat)) + add     (OIDN_NORM_RMS: mean(g) left out)
 *   dweight = sum of dy hat over the rows,  dshift = sum of dy
 * add (m x n or NULL) is what else reaches x.  dx, dweight and dshift may each
 * be NULL.  Nothing is kept from the forward pass but x. */
int oidn_norm_backward_workspace_bytes(long m, int n, int dtype, size_t* bytes);
int oidn_norm_backward(const void* dy, long lddy, const void* x, long ldx, const float* weight,
                       const void* add, long ldadd, void* dx, long lddx, float* dweight, float* dshift,
                       long m, int n, int norm, float eps, int dtype, void* workspace, size_t ws_bytes,
                       hipStream_t stream);

/* After a block with the output o, and before the next one:
 *   u = scale x + gate drop(norm(o) weight + shift)
 *   v = next_norm(u) next_weight + next_shift        (of u as stored)
 * gate: NULL (1), or a row of n floats at pitch ldg for every gate_rows rows (an
 * image, a sequence; the last may be short).  drop: oidn_dropout's with p and rng
 * (p = 0: none; rng unused).  norm may be OIDN_NORM_NONE (a block that norms only
 * its input); next_norm too, with v NULL.  Vectors may be NULL: 1 and 0. */
int oidn_norm_residual(const void* o, long ldo, const float* weight, const float* shift, const float* gate,
                       long ldg, long gate_rows, const void* x, long ldx, float scale, float p,
                       const unsigned long long* rng, void* u, long ldu, const float* next_weight,
                       const float* next_shift, void* v, long ldv, long m, int n, int norm, int next_norm,
                       float eps, int dtype, hipStream_t stream);

/* Its gradients, from dv and from du, what else reaches u (NULL: nothing):
 *   D = du + next_norm'(dv; u),  dx = scale D,
 *   dgate = sum of D drop(norm(o) weight + shift) over the gate's rows,
 *   h = drop(D gate),  dweight = sum of h norm(o),  dshift = sum of h,
 *   d_o = norm'(h weight; o),
 *   dnext_weight = sum of dv next_norm(u),  dnext_shift = sum of dv
 * D is not rounded on the way.  u as oidn_norm_residual stored it (unused with
 * next_norm OIDN_NORM_NONE, where dv is NULL and du is not); o, vectors, gate, p and
 * rng's contents as given to it: the mask is formed again, not stored.  Any result
 * may be NULL.  gate_rows of the size call: 0 without a gate. */
int oidn_norm_residual_backward_workspace_bytes(long m, int n, long gate_rows, int dtype, size_t* bytes);
int oidn_norm_residual_backward(const void* du, long lddu, const void* dv, long lddv, const void* o,
                                long ldo, const float* weight, const float* shift, const float* gate,
                                long ldg, long gate_rows, const void* u, long ldu, float scale, float p,
                                const unsigned long long* rng, const float* next_weight, void* dx, long lddx,
                                void* d_o, long lddo, float* dgate, long lddg, float* dweight, float* dshift,
                                float* dnext_weight, float* dnext_shift, long m, int n, int norm,
                                int next_norm, float eps, int dtype, void* workspace, size_t ws_bytes,
                                hipStream_t stream);

/* Dropout:  y = drop(x) + residual  (residual m x n or NULL).  Its gradient is
 * the same call on dy without the residual.  The mask is never stored: with
 * t = rint(65536 p), element (i, j) is kept, times 65536 / (65536 - t), where its 16
 * bits are >= t, else 0 whatever it holds.  The bits are those of Philox4x32-10 with
 * the 64-bit key rng[0] (the seed) and the counter (i ceil(n / 8) + j / 8, rng[1]),
 * both 64 bits, low words first: element j % 8 = 2 w + b takes half b of word w
 * (0: low).  So they depend on the element's place, seed and offset alone, not on
 * pitch or type.  rng: two 64-bit words in device memory, read by the kernel, so
 * that a captured graph drops other elements at each replay if the program (or a node of
 * the graph) changes rng[1] in between; calls that are to be independent take
 * different offsets.  p in [0, 1]; p = 0: nothing is dropped and rng may be NULL. */
int oidn_dropout(const void* x, long ldx, const void* residual, long ldr, void* y, long ldy, long m, int n,
                 float p, const unsigned long long* rng, int dtype, hipStream_t stream);

/* Measurement helper, not part of the denoise path: `blocks` workgroups of
 * 4 waves, each wave issuing iters x 8 independent 16x16x32 MFMAs (fp16, or
 * bf16 with dtype OIDN_BF16) with no memory traffic, to measure the matrix
 * rate the device sustains.  *flops receives the launch's work (2 per
 * multiply-add).  sink: a device buffer of at least 256 floats (written
 * only in a case the operands never produce).  Enqueued on `stream`. */
int oidn_calibrate_mfma(int dtype, long iters, int blocks, float* sink, long long* flops,
                        hipStream_t stream);

/* Measurement helper, not part of the denoise path: reads the `bytes` of
 * device buffer `buf` once (16-byte streaming loads, 2048 workgroups), to
 * measure the HBM read rate.  bytes: a multiple of 16; sink: a device buffer
 * of at least 256 floats (written only in a case the data never produces). */
int oidn_calibrate_read(const void* buf, size_t bytes, float* sink, hipStream_t stream);

/* Timing helpers: a hipEvent_t with timing enabled, its destruction, and the
 * milliseconds between two completed events (synchronises on `end`). */
int oidn_event_create(void** event);
int oidn_event_destroy(void* event);
int oidn_event_elapsed_ms(void* start, void* end, float* ms);

#ifdef __cplusplus
}
#endif

#endif /* OIDN_MI355X_H */
