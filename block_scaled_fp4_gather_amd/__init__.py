"""Block-scaled FP4 (MXFP4 / NVFP4) mixture-of-experts layer for AMD MI355X.

The compute path is the HIP library ``libmoe_fp4.so`` built from ``csrc/``;
``moe`` is its thin ctypes binding (argument marshalling only): ``Desc``
(shape, weight format, activation format "bf16" / "mxfp8", activation
function), ``Fp4MoE`` (prepared weights + workspace, callable), and the
entry points one to one.  ``block`` binds the operators around the layer
(``Router``, ``Fp8Linear``, ``block_norm``) and joins them in ``Fp4MoEBlock``.
``experts`` makes FP4 weights (``fp4_quantize``), multiplies by them with FP4
activations (``Fp4Linear``), and trains bf16 experts: ``group_routes``,
``gather_routes``, ``grouped_linear``, ``combine_routes``, with gradients.
``synth`` draws seeded synthetic inputs.
"""
