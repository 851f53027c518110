"""One attention layer of a quantized decoder, a token per sequence at a time:

  x -> QGemmDyn (q, k and v) -> kv_append (rotary positions, int8 pages)
    -> paged_attention (weights added to the scores) -> QGemmDyn (output)

and, when a sequence reaches its capacity, kv_evict into fresh pages.  Run as
a module it decodes a few tokens with random weights:

    python -m int8_quantized_gb300.decode
"""
import torch

import int8_quantized_gb300 as q


class DecodeAttention:
    """Weights are int8 [in, out] with a scale per output column (typeB
    I8Q_S8 of QGemmDyn): w_qkv [hidden, (q_heads + 2 kv_heads) * head_dim],
    w_out [q_heads * head_dim, hidden].  cos, sin: fp32 [positions, pairs].

    A sequence that holds `capacity` tokens is cut to `budget` before its next
    token: the first `sink`, the last `recent` and the most attended others.
    """

    def __init__(self, w_qkv, w_qkv_scale, w_out, w_out_scale, cos, sin, *, sequences, q_heads, kv_heads, head_dim,
                 capacity, budget, sink=4, recent=32, page_size=16):
        if not 0 < budget < capacity:
            raise ValueError("budget must be below capacity")
        if sink < 0 or recent < 0 or sink + recent > budget:
            raise ValueError("sink + recent must be within 0 .. budget")
        dev = w_qkv.device
        self.B, self.Hq, self.H, self.D = sequences, q_heads, kv_heads, head_dim
        self.capacity, self.budget, self.sink, self.recent, self.page = capacity, budget, sink, recent, page_size
        hidden, width = w_qkv.shape
        self.qkv_gemm = q.QGemmDyn(sequences, width, hidden, q.BF16, q.S8, q.BF16, bias=False)
        self.qkv_gemm.set_params(w_qkv, w_qkv_scale)
        self.out_gemm = q.QGemmDyn(sequences, hidden, q_heads * head_dim, q.BF16, q.S8, q.BF16, bias=False)
        self.out_gemm.set_params(w_out, w_out_scale)
        self.cos, self.sin = cos, sin
        per = -(-capacity // page_size)
        pages = sequences * per + -(-budget // page_size)  # one sequence at a time moves into the spare pages
        shape = (pages, kv_heads, page_size, head_dim)
        k, scale = torch.zeros(shape, dtype=torch.int8, device=dev), torch.ones(shape[:3], device=dev)
        self.cache = q.KVCache(k, torch.zeros_like(k), scale, scale.clone(), torch.zeros_like(scale))
        self.free = list(range(pages))
        self.table = torch.full((sequences, per), -1, dtype=torch.int32, device=dev)
        self.owned = [[] for _ in range(sequences)]
        self.length = [0] * sequences
        self.position = [0] * sequences                # of the next token; eviction does not change it
        self.seq = torch.arange(sequences, dtype=torch.int32, device=dev)
        self.qkv = torch.empty((sequences, width), dtype=torch.bfloat16, device=dev)
        self.attended = torch.empty((sequences, q_heads, head_dim), dtype=torch.bfloat16, device=dev)
        self.workspace = torch.empty(q.paged_attention_workspace_size(self.cache, self.table, q_heads, True),
                                     dtype=torch.uint8, device=dev)

    def _grow(self, b):
        if self.length[b] == len(self.owned[b]) * self.page:
            self.owned[b].append(self.free.pop())
            self.table[b, len(self.owned[b]) - 1] = self.owned[b][-1]

    def evict(self, b):
        """Cut sequence b to its budget; returns the kept tokens' indices [kv_heads, budget]."""
        dev = self.table.device
        need = -(-self.budget // self.page)
        new = self.free[-need:]
        new_table = torch.tensor([new], dtype=torch.int32, device=dev)
        kept = torch.empty((1, self.H, self.budget), dtype=torch.int32, device=dev)
        q.kv_evict(self.cache, self.table[b:b + 1], torch.tensor([self.length[b]], dtype=torch.int32, device=dev),
                   new_table, kept, sink=self.sink, recent=self.recent)
        self.free = self.free[:-need] + self.owned[b]
        self.owned[b], self.length[b] = new, min(self.length[b], self.budget)
        self.table[b].fill_(-1)
        self.table[b, :need] = new_table[0]
        return kept[0]

    def step(self, x, out):
        """x, out: bf16 [sequences, hidden], the next token of every sequence."""
        dev = x.device
        if max(self.position) >= self.cos.shape[0]:
            raise ValueError("a sequence has no position left in cos and sin")
        for b in range(self.B):
            if self.length[b] == self.capacity:
                self.evict(b)
            self._grow(b)
        self.qkv_gemm.forward(x, self.qkv)
        rows = self.qkv.view(self.B, self.Hq + 2 * self.H, self.D)
        query, key, value = rows.split((self.Hq, self.H, self.H), 1)
        index = torch.tensor(self.length, dtype=torch.int32, device=dev)
        positions = torch.tensor(self.position, dtype=torch.int32, device=dev)
        q.kv_append(self.cache, self.table, self.seq, index, key, value, q=query, q_out=query, positions=positions,
                    cos=self.cos, sin=self.sin)
        q.paged_attention(self.cache, self.table, index + 1, query, self.attended, accumulate=True,
                          workspace=self.workspace)
        self.out_gemm.forward(self.attended.view(self.B, -1), out)
        self.length = [n + 1 for n in self.length]
        self.position = [n + 1 for n in self.position]
        return out


def random_layer(sequences=4, hidden=1024, q_heads=16, kv_heads=4, head_dim=64, capacity=96, budget=64, positions=4096,
                 seed=0, device="cuda", sink=None, recent=None):
    """A DecodeAttention with random weights; sink and recent: 4 and 32, or what the budget has room for."""
    sink = min(4, budget) if sink is None else sink
    recent = min(32, budget - sink) if recent is None else recent
    g = torch.Generator(device=device)
    g.manual_seed(seed)

    def weight(rows, columns):
        w = torch.randint(-127, 128, (rows, columns), generator=g, device=device, dtype=torch.int8)
        return w, torch.full((columns,), 1.0 / (73.0 * rows ** 0.5), device=device)

    pairs = head_dim // 2
    turn = torch.arange(positions, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(pairs) / pairs)
    return DecodeAttention(*weight(hidden, (q_heads + 2 * kv_heads) * head_dim), *weight(q_heads * head_dim, hidden),
                           turn.cos().float().to(device), turn.sin().float().to(device), sequences=sequences,
                           q_heads=q_heads, kv_heads=kv_heads, head_dim=head_dim, capacity=capacity, budget=budget,
                           sink=sink, recent=recent)


def main():
    layer = random_layer()
    x = torch.randn((layer.B, 1024), device="cuda").to(torch.bfloat16)
    out = torch.empty_like(x)
    for step in range(200):
        layer.step(x, out)
        x.copy_(torch.nn.functional.normalize(out.float(), dim=-1) * 32)
        if step % 50 == 49:
            print(f"step {step + 1}: cached {layer.length}, output rms {out.float().square().mean().sqrt():.4f}")
    q.sync_status()


if __name__ == "__main__":
    main()
